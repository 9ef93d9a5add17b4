"""How the attention's work is shared: units of work over CTAs, restated, over many shapes of
batches.  Every CTA between the one that holds a cut block's first tile and the one that
holds its last holds a tile of the block, which the joins count on."""
import random

TILE_BOTH, TILE_ONE, BLOCK_COST, MIN_SHARE, CTAS = 4, 3, 10, 12, 152


def shares(units):
    n = max(1, min(CTAS, -(-units // MIN_SHARE)))
    each, extra = divmod(units, n)
    return [each * c + min(c, extra) for c in range(n + 1)]


def test_shares_are_never_less_than_a_tile():
    least = min(min(b - a for a, b in zip(s, s[1:]))
                for s in map(shares, range(BLOCK_COST + TILE_ONE, 5000)))
    assert least == (MIN_SHARE + 1) // 2 and least >= TILE_BOTH


def test_every_cta_of_a_cut_block_has_a_tile():
    r = random.Random(1)
    for _ in range(300):
        H = r.choice([1, 2, 3, 8])
        blocks = [(r.choice([TILE_BOTH, TILE_ONE]), 1 + int(r.expovariate(1 / r.choice([1, 5, 200]))))
                  for _ in range(r.choice([1, 2, 9, 60]))]
        items, u = [], 0                                   # (first unit of each tile) per (block, head)
        for per, n in blocks:
            for _ in range(H):
                items.append([u + BLOCK_COST + per * j for j in range(n)])
                u += BLOCK_COST + per * n
        begin = shares(u)
        of = lambda x: next(c for c in range(len(begin) - 1) if begin[c] <= x < begin[c + 1])
        for tiles in items:
            who = [of(t) for t in (tiles if len(tiles) < 60 else tiles[::20] + tiles[-1:])]
            if len(tiles) < 60:
                assert sorted(set(who)) == list(range(who[0], who[-1] + 1))
            else:
                c0, c1 = who[0], who[-1]
                for c in range(c0 + 1, c1):
                    assert any(begin[c] <= t < begin[c + 1] for t in tiles), (begin[c], begin[c + 1])
