"""The oracle of the chunk operators, held against what their definitions fix."""
import numpy as np
import pytest

import oracle
from oracle import chunk as oc


def rng(*key):
    return np.random.default_rng([11, *key])


def test_whole_prompt_rows_are_dense_causal_attention():
    g = rng(1)
    n, G, D = 37, 2, 8
    q = g.standard_normal((n, G, D))
    k, v = g.standard_normal((2, n, D))
    out, lse = oc.chunk_attend(q, k, v, 0, 0.3)
    for i in range(n):
        o, z = oracle.attend(q[i], k[:i + 1], v[:i + 1], 0.3)
        assert np.allclose(out[i], o, atol=1e-12) and np.allclose(lse[i], z, atol=1e-12)


def test_chunks_join_to_the_whole_prompt():
    g = rng(2)
    n, D = 50, 8
    q = g.standard_normal((n, 1, D))
    k, v = g.standard_normal((2, n, D))
    whole, z = oc.chunk_attend(q, k, v, 0, 1.0, window=9, sink=2)
    for cut in (1, 13, 49):
        a = oc.chunk_attend(q[:cut], k[:cut], v[:cut], 0, 1.0, window=9, sink=2)
        b = oc.chunk_attend(q[cut:], k, v, cut, 1.0, window=9, sink=2)
        assert np.allclose(np.concatenate([a[0], b[0]]), whole, atol=1e-12)
        assert np.allclose(np.concatenate([a[1], b[1]]), z, atol=1e-12)


def test_window_and_sink_by_hand():
    k = np.zeros((6, 4))
    v = np.arange(6.0)[:, None] * np.ones((6, 4))
    out, lse = oc.chunk_attend(np.ones((1, 1, 4)), k, v, 5, 1.0, window=2, sink=1)
    assert np.allclose(out[0, 0], (0 + 4 + 5) / 3) and np.isclose(lse[0, 0], np.log(3))
    out, lse = oc.chunk_attend(np.ones((2, 1, 4)), k, v, -1, 1.0)      # refused rows see nothing
    assert np.all(out == 0) and np.all(np.isneginf(lse))
    out, _ = oc.chunk_attend(np.ones((1, 1, 4)), k, v, 5, 1.0, absent=[4, 5])
    assert np.allclose(out[0, 0], 1.5)


def pool(num_pages, ctx, maxp=8):
    """Sequences holding just the pages their tokens need, taken from a full stack."""
    p = oc.Pool(num_pages, len(ctx), maxp)
    for b, c in enumerate(ctx):
        for i in range(-(-c // 16)):
            p.block_table[b, i] = p.free.pop()
        p.n_pages[b] = -(-c // 16)
        p.ctx[b] = c
    return p


def test_plan_by_hand():
    p = pool(10, [16, 0, 5])
    assert p.free == list(range(9, 1, -1))[:8]
    start, seq, pos, slot, flags = oc.plan(p, [1, 17, 11], 32)
    assert flags == 0
    assert list(start) == [0, 1, 18, 29]
    assert list(p.block_table[0, :2]) == [0, 2] and list(p.block_table[1, :2]) == [3, 4]
    assert list(p.n_pages) == [2, 2, 1]
    assert slot[0] == 2 * 16 and pos[0] == 16
    assert list(slot[1:18]) == list(range(48, 65)) and list(pos[18:29]) == list(range(5, 16))
    assert list(slot[18:29]) == [16 + i for i in range(5, 16)]
    assert list(seq[28:]) == [2, -1, -1, -1] and list(slot[29:]) == [-1] * 3
    again = oc.plan(p, [1, 17, 11], 32)
    assert np.array_equal(again[3], slot) and len(p.free) == 5


def test_plan_serves_in_order_and_needless_requests_always():
    p = pool(5, [16, 16, 1])                       # 2 free
    start, seq, pos, slot, flags = oc.plan(p, [16, 32, 15], 64)
    assert flags == oc.CAPACITY
    assert np.all(slot[:16] >= 0) and np.all(slot[16:48] == -1) and np.all(pos[16:48] == -1)
    assert np.all(slot[48:63] >= 0)
    assert list(p.n_pages) == [2, 1, 1] and len(p.free) == 1


def test_release_undoes_a_plan():
    p = pool(20, [3, 40, 0, 17])
    before = list(p.free)
    held = [list(p.block_table[b, :p.n_pages[b]]) for b in range(4)]
    oc.release(p, [0, 1, 0, 1])
    assert list(p.n_pages) == [1, 0, 0, 0] and list(p.ctx) == [3, 0, 0, 0]
    assert p.free == before + (held[1] + held[3])[::-1]
    oc.plan(p, [0, 40, 0, 17], 64)
    assert [list(p.block_table[b, :p.n_pages[b]]) for b in range(4)] == held


@pytest.mark.parametrize("ctx,n", [(0, 40), (15, 1), (5, 30), (16, 16)])
def test_append_summaries_are_those_of_the_whole_page(ctx, n):
    g = rng(3, ctx, n)
    p = pool(8, [ctx])
    k, v = np.zeros((2, 8, 2, 16, 4))
    meta = np.full((1, 8, 2, 2, 4), 99.0)
    allk = g.standard_normal((ctx + n, 2, 4))
    if ctx:
        q = pool(8, [0])
        s = oc.plan(q, [ctx], ctx)
        oc.append(q, k, v, meta, allk[:ctx], allk[:ctx], *s[:4])
    s = oc.plan(p, [n], n)
    oc.append(p, k, v, meta, allk[ctx:], -allk[ctx:], *s[:4])
    assert p.ctx[0] == ctx + n
    for pg in range(-(-(ctx + n) // 16)):
        rows = allk[16 * pg:16 * pg + 16]
        assert np.array_equal(meta[0, pg, :, 0], rows.min(0))
        assert np.array_equal(meta[0, pg, :, 1], rows.max(0))
        assert np.array_equal(k[p.block_table[0, pg], :, :len(rows)], rows.transpose(1, 0, 2))
