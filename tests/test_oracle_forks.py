"""Pins of the fork and truncation oracle: pages are counted as they are held, no sequence's content
changes by what another does."""
import numpy as np
import pytest

from oracle import chunk as oc
from oracle import forks as of


def check_counts(pool, refs):
    held = np.zeros(pool.num_pages, dtype=int)
    for b in range(len(pool.n_pages)):
        for p in pool.block_table[b, :pool.n_pages[b]]:
            held[p] += 1
        if pool.ctx[b] % oc.PAGE:                                 # the last page is its own
            assert refs[pool.block_table[b, pool.ctx[b] // oc.PAGE]] == 0
    assert np.array_equal(np.array(refs), np.maximum(held - 1, 0))
    assert sorted(pool.free) == sorted(np.flatnonzero(held == 0).tolist())


class Mirror:
    """What each sequence should hold, kept apart: a list of token numbers."""

    def __init__(self, batch):
        self.seqs = [[] for _ in range(batch)]
        self.count = 0

    def grow(self, b, n):
        self.seqs[b] += range(self.count + 1, self.count + n + 1)
        self.count += n


def step(g, pool, refs, mirror, k, v, meta):
    """One random step: new tokens, forks into empty sequences, cuts."""
    B = len(pool.ctx)
    new = g.integers(0, 40, B) * (g.random(B) < 0.5)
    start, seq, pos, slot, _ = oc.plan(pool, new, int(new.sum()))
    for b in range(B):
        n = int((slot[seq == b] >= 0).sum())
        mirror.grow(b, n)
    rows = np.array([mirror.seqs[b][p] if s >= 0 else 0 for b, p, s in zip(seq, pos, slot)], float)
    x = rows[:, None, None] * np.ones((1, k.shape[1], k.shape[3]))
    oc.append(pool, k, v, meta, x, -x, start, seq, pos, slot)
    src = np.full(B, -1)
    empty = np.flatnonzero(pool.n_pages == 0)
    full = np.flatnonzero(pool.n_pages > 0)
    if len(full):
        for b in empty:
            if g.random() < 0.7:
                src[b] = g.choice(full)
    fs, fp, _ = of.fork(pool, refs, src)
    of.carry(pool, k, v, meta, fs, fp)
    for b in np.flatnonzero(fs >= 0):
        mirror.seqs[b] = list(mirror.seqs[fs[b]])
    keep = np.where(g.random(B) < 0.5, (pool.ctx * g.random(B)).astype(int), -1)
    keep[g.random(B) < 0.15] = 0
    before = pool.ctx.copy()
    fs, fp, flags = of.truncate(pool, refs, keep)
    of.carry(pool, k, v, meta, fs, fp)
    for b in range(B):
        if keep[b] >= 0 and pool.ctx[b] == min(keep[b], before[b]):
            mirror.seqs[b] = mirror.seqs[b][:keep[b]]


def check_contents(pool, mirror, k, v, meta):
    for b, want in enumerate(mirror.seqs):
        assert pool.ctx[b] == len(want)
        for lp in range(-(-len(want) // oc.PAGE)):
            rows = np.array(want[lp * 16:lp * 16 + 16], float)
            page = pool.block_table[b, lp]
            assert np.array_equal(k[page, 0, :len(rows), 0], rows)
            assert np.array_equal(v[page, -1, :len(rows), -1], -rows)
            assert meta[b, lp, 0, 0, 0] == rows.min() and meta[b, lp, 0, 1, 0] == rows.max()


@pytest.mark.parametrize("batch,pages", [(2, 9), (5, 30), (12, 60)])
def test_random_steps_leave_every_sequence_its_own(batch, pages):
    g = np.random.default_rng([7, batch])
    pool, refs, mirror = oc.Pool(pages, batch, 12), [0] * pages, Mirror(batch)
    k, v = np.zeros((2, pages, 1, 16, 2))
    meta = np.zeros((batch, 12, 1, 2, 2))
    shared = 0
    for _ in range(60):
        step(g, pool, refs, mirror, k, v, meta)
        check_counts(pool, refs)
        check_contents(pool, mirror, k, v, meta)
        shared = max(shared, max(refs))
    assert shared >= 1 or batch == 2             # two sequences seldom get to share a full page here


def test_a_truncation_to_nothing_is_a_release():
    a, b = (oc.Pool(20, 3, 8) for _ in range(2))
    for p in (a, b):
        oc.plan(p, [40, 17, 100], 157)
        p.ctx[:] = 40, 17, 100
    of.truncate(a, None, [0, -1, 0])
    oc.release(b, np.array([1, 0, 1]))
    assert a.free == b.free and a.n_pages.tolist() == b.n_pages.tolist()


def test_a_source_whose_last_page_does_not_exist_costs_no_page():
    pool, refs = oc.Pool(10, 4, 4), [0] * 10
    oc.plan(pool, [20, 20, 0, 0], 40)
    pool.ctx[:2] = 20
    pool.block_table[0, 1] = 10
    fs, fp, flags = of.fork(pool, refs, [-1, -1, 0, 1])
    assert flags == of.BAD_INDEX and fs.tolist() == [-1, -1, -1, 1] and pool.n_pages.tolist() == [2, 2, 0, 2]
    assert len(pool.free) == 5 and sum(refs) == 1
