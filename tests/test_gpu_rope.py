"""GPU parity of the rotation and of the append that applies it: values within bounds derived from the
roundings, everything else exactly."""
import math

import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from oracle import rope as R
from tests.test_gpu_chunk import both_pools, i32, plan_both

pytestmark = pytest.mark.gpu
MARK = 777.0                                      # what outputs hold before a call
BAD_INDEX = 1


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def bf16(g, *shape, scale=1.0):
    x = torch.from_numpy(g.standard_normal(shape).astype(np.float32) * np.float32(scale))
    return x.bfloat16().cuda()


def marked(*shape):
    return torch.full(shape, MARK, dtype=torch.bfloat16, device="cuda")


def make(g, rot, dim, layout, norm, amp=None, base=1e4, **kw):
    qw, kw_ = ((1 + 0.3 * bf16(g, dim)) if n else None for n in norm)
    return se.Rope.make(rot, base, layout=layout, q_weight=qw, k_weight=kw_, amplitude=amp, **kw)


def f64(x):
    return x.double().cpu().numpy()


def check(rope, x, got, pos, weight, before):
    """Rows with a position against the oracle, the others against what was there."""
    turns = [] if rope.turns is None else [t % 2 ** 64 for t in rope.turns.tolist()]
    w = None if weight is None else f64(weight)
    amp = float(np.float32(rope.amplitude))
    eps = float(np.float32(rope.eps))
    want = R.rotate(f64(x), pos, turns, amp, rope.layout, w, eps)
    room = R.rounding_bound(f64(x), want, 2 * len(turns), amp, rope.layout, w, eps)
    live = np.asarray(pos) >= 0
    off = np.abs(f64(got) - want)[live] - room[live]
    assert off.size == 0 or off.max() <= 0, off.max()
    assert np.array_equal(f64(got)[~live], f64(before)[~live])


def small_ws():
    return se.workspace(se.se_small_workspace())


@pytest.mark.parametrize("rows,hq,hk,dim,rot,layout,norm", [
    (1, 1, 1, 64, 64, 0, (1, 1)), (1, 32, 4, 128, 128, 0, (1, 1)), (1, 33, 3, 128, 128, 1, (0, 1)),
    (2, 5, 7, 64, 16, 1, (1, 0)), (7, 9, 2, 128, 96, 0, (1, 1)), (7, 4, 4, 128, 112, 1, (0, 0)),
    (64, 32, 4, 128, 64, 0, (1, 1)), (65, 8, 8, 64, 48, 1, (0, 0)), (300, 16, 1, 128, 128, 0, (1, 1)),
    (301, 3, 0, 64, 32, 0, (1, 1)), (5, 0, 6, 128, 128, 0, (1, 1)), (9, 4, 2, 64, 0, 0, (1, 1)),
    (3, 1024, 2, 64, 64, 1, (1, 1)), (2500, 6, 2, 128, 32, 1, (0, 1))])
def test_rows_of_every_shape(rows, hq, hk, dim, rot, layout, norm):
    g = np.random.default_rng([11, rows, hq, dim, rot])
    rope = make(g, rot, dim, layout, norm, amp=1.25 if rows % 2 else None)
    pos = g.integers(0, 1 << 20, rows)
    pos[::5] = [0, 1, 2 ** 30 - 1, 2 ** 31 - 1, 17][rows % 5]
    if rows > 2:
        pos[1] = -1
    q, k = (bf16(g, rows, h, dim, scale=3) if h else None for h in (hq, hk))
    qo, ko = (None if x is None else marked(*x.shape) for x in (q, k))
    ws = small_ws()
    se.se_qk_rope(rope, i32(pos), q, k, qo, ko, ws)
    for x, out, w in ((q, qo, rope.q_weight), (k, ko, rope.k_weight)):
        if x is not None:
            check(rope, x, out, pos, w, marked(*x.shape))
    assert se.status_word(ws) == 0


def test_no_rows():
    g = np.random.default_rng(1)
    rope = make(g, 64, 64, 0, (1, 1))
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    se.se_qk_rope(rope, i32([]), q, None, q.clone(), None, small_ws())


def test_slices_of_packed_rows_and_in_place():
    """q and k out of packed rows, written back over themselves: v and what lies between stay."""
    g = np.random.default_rng(12)
    rope = make(g, 128, 128, 0, (1, 1))
    rows, hq, hk, d = 37, 8, 2, 128
    x = bf16(g, rows, hq + 2 * hk + 1, d)
    before = x.clone()
    pos = g.integers(-1, 5000, rows)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    se.se_qk_rope(rope, i32(pos), q, k, q, k, small_ws())
    check(rope, before[:, :hq], q, pos, rope.q_weight, before[:, :hq])
    check(rope, before[:, hq:hq + hk], k, pos, rope.k_weight, before[:, hq:hq + hk])
    assert x[:, hq + hk:].equal(before[:, hq + hk:])
    # one of them alone, into a slice of other rows
    out = marked(rows, hq + 3, d)
    se.se_qk_rope(rope, i32(pos), before[:, :hq], None, out[:, 2:2 + hq], None, small_ws())
    assert out[:, 2:2 + hq][torch.from_numpy(pos >= 0)].equal(q[torch.from_numpy(pos >= 0)])
    assert (out[:, :2] == MARK).all() and (out[:, 2 + hq:] == MARK).all()


def test_values_that_are_no_numbers_stay_in_their_head():
    g = np.random.default_rng(13)
    rope = make(g, 64, 128, 1, (1, 1))
    x = bf16(g, 6, 5, 128)
    clean = marked(6, 5, 128)
    se.se_qk_rope(rope, i32(range(6)), x, None, clean, None, small_ws())
    for bad in (math.nan, math.inf, -math.inf):
        y, out = x.clone(), marked(6, 5, 128)
        y[2, 3, 100] = bad
        se.se_qk_rope(rope, i32(range(6)), y, None, out, None, small_ws())
        assert out[2, 3, 100].isnan()
        out[2, 3] = clean[2, 3]
        assert out.equal(clean)
    # without a norm only the pair is touched
    plain = make(g, 128, 128, 1, (0, 0))
    y, out = x.clone(), marked(6, 5, 128)
    se.se_qk_rope(plain, i32(range(6)), x, None, clean, None, small_ws())
    y[2, 3, 100] = math.nan
    se.se_qk_rope(plain, i32(range(6)), y, None, out, None, small_ws())
    assert out[2, 3, 100:102].isnan().all()
    out[2, 3, 100:102] = clean[2, 3, 100:102]
    assert out.equal(clean)


def test_extremes_of_the_norm():
    """Rows of zeros, of the smallest and of large values (their squares within fp32)."""
    g = np.random.default_rng(14)
    rope = make(g, 64, 64, 0, (1, 1))
    x = bf16(g, 4, 2, 64)
    x[0] = 0
    x[1] *= 2.0 ** -126
    x[2] *= 2.0 ** 55
    out = marked(4, 2, 64)
    pos = [0, 3, 70000, 5]
    se.se_qk_rope(rope, i32(pos), x, None, out, None, small_ws())
    assert (out[0] == 0).all()
    check(rope, x[2:], out[2:], pos[2:], rope.q_weight, out[2:])
    # squares below fp32's range count as 0: x / sqrt(eps), to a part in 2^-8 and the smallest steps
    check(rope, x[1:2], out[1:2], pos[1:2], rope.q_weight, out[1:2])


@pytest.mark.parametrize("scaling,low,high", [(1, 1, 4), (2, 1, 4), (3, 1, 32), (4, 1, 4)])
def test_scaled_frequencies_at_far_positions(scaling, low, high):
    """Against angles of the formula in 64 bits (the frequencies' own error: 2^-52 of an angle of 2^20)."""
    g = np.random.default_rng([15, scaling])
    rope = make(g, 96, 128, 0, (0, 0), base=5e5, scaling=scaling, factor=8.0, original_len=8192.0, low=low,
                high=high)
    f, amp = R.frequencies(5e5, 96, scaling, 8.0, 8192.0, low, high)
    x, pos = bf16(g, 50, 3, 128), g.integers(0, 1 << 20, 50)
    out = marked(50, 3, 128)
    se.se_qk_rope(rope, i32(pos), x, None, out, None, small_ws())
    angle = pos[:, None].astype(np.float64) * np.array(f)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y = f64(x)
    want = y.copy()
    want[..., :48] = amp * (y[..., :48] * c - y[..., 48:96] * s)
    want[..., 48:96] = amp * (y[..., 48:96] * c + y[..., :48] * s)
    room = R.rounding_bound(y, want, 96, amp, 0, None, 0)
    assert (np.abs(f64(out) - want) <= room).all()


# ---------------------------------------------------------------------------
# the append
# ---------------------------------------------------------------------------

def cache(g, pages, batch, maxp, heads, dim, summaries, table, ctx):
    k, v = bf16(g, pages, heads, 16, dim), bf16(g, pages, heads, 16, dim)
    meta = bf16(g, batch, maxp, heads, 2, dim).sort(3).values.contiguous() if summaries else None
    return se.PagedKV(k, v, meta, table, ctx)


def copy_of(kv):
    return se.PagedKV(kv.k.clone(), kv.v.clone(), None if kv.meta is None else kv.meta.clone(),
                      kv.block_table, kv.ctx_len.clone())


def append_both(kv, rope, q, k, v, chunk, batch, flags=0):
    """The one call against se_qk_rope and se_kv_append_chunk: the same bits everywhere."""
    two, rows = copy_of(kv), k.shape[0]
    qo, q2 = (None if q is None else marked(rows, q.shape[1], q.shape[2]) for _ in range(2))
    k2 = k.clone()
    se.se_qk_rope(rope, chunk.pos, q, k, q2, k2, small_ws())
    ws2 = small_ws()
    se.se_kv_append_chunk(two, k2.contiguous(), v.contiguous(), chunk, batch, ws2)
    ws = small_ws()
    se.se_rope_append_chunk(kv, rope, q, k, v, qo, chunk, batch, ws)
    assert se.status_word(ws) == se.status_word(ws2) == flags
    assert kv.k.equal(two.k) and kv.v.equal(two.v) and kv.ctx_len.equal(two.ctx_len)
    assert kv.meta is None or kv.meta.equal(two.meta)
    assert q is None or qo.equal(q2)
    return qo


CASES = [(1, 1, 1, 1, 64, 64, 0, 1), (5, 17, 8, 2, 128, 128, 0, 1), (5, 40, 4, 4, 128, 64, 1, 0),
         (64, 1, 32, 4, 128, 128, 0, 1), (9, 150, 8, 8, 64, 48, 1, 0), (3, 700, 16, 1, 64, 64, 0, 1),
         (200, 9, 4, 2, 64, 32, 0, 1), (2, 3000, 8, 4, 128, 128, 0, 1), (33, 16, 6, 3, 128, 0, 0, 1)]


@pytest.mark.parametrize("batch,hi,hq,hk,dim,rot,layout,norm", CASES)
def test_append_is_rotation_then_append(batch, hi, hq, hk, dim, rot, layout, norm):
    g = np.random.default_rng([16, batch, hi, dim])
    maxp = 3 * (hi // 16 + 2)
    pages = batch * maxp
    o, p = both_pools(pages, batch, maxp)
    order = g.permutation(pages).tolist()
    o.free = list(order)
    p.free_pages.copy_(i32(order))
    ws = se.workspace(se.se_page_pool_workspace(batch))
    rope = make(g, rot, dim, layout, (norm, norm))
    kv = cache(g, pages, batch, maxp, hk, dim, hi % 2 == 1, p.block_table, p.ctx_len)
    for step in range(3):
        new = g.integers(0, hi + 1, batch)
        new[g.random(batch) < 0.3] = 1
        rows = int(new.sum()) + step * 5
        chunk = plan_both(o, p, new, rows, ws)
        x = bf16(g, rows, hq + 2 * hk, dim)
        q = x[:, :hq] if step != 1 else None
        append_both(kv, rope, q, x[:, hq:hq + hk], x[:, hq + hk:], chunk, batch)
        o.ctx += new
        assert p.ctx_len.cpu().tolist() == o.ctx.tolist()


def test_append_in_place_and_rows_behind_the_last_sequence():
    g = np.random.default_rng(17)
    o, p = both_pools(40, 3, 10)
    rope = make(g, 128, 128, 0, (1, 1))
    ws = se.workspace(se.se_page_pool_workspace(3))
    kv = cache(g, 40, 3, 10, 2, 128, True, p.block_table, p.ctx_len)
    chunk = plan_both(o, p, [20, 0, 33], 60, ws)
    x = bf16(g, 60, 12, 128)
    before, other = x.clone(), copy_of(kv)
    out = append_both(other, rope, x[:, :8], x[:, 8:10], x[:, 10:], chunk, 3)
    assert x.equal(before) and (out[53:] == MARK).all()
    se.se_rope_append_chunk(kv, rope, x[:, :8], x[:, 8:10], x[:, 10:], x[:, :8], chunk, 3, small_ws())
    assert x[:53, :8].equal(out[:53]) and x[53:].equal(before[53:]) and x[:, 8:].equal(before[:, 8:])
    assert kv.k.equal(other.k) and kv.meta.equal(other.meta)


def test_append_with_holes_and_bad_rows():
    """Rows without a page between others, slots, sequences and positions that do not exist: as the two
    calls take them."""
    g = np.random.default_rng(18)
    for trial in range(12):
        batch, rows, maxp = 3, 70, 6
        o, p = both_pools(18, batch, maxp)
        ws = se.workspace(se.se_page_pool_workspace(batch))
        rope = make(g, 64, 64, trial % 2, (1, 1))
        kv = cache(g, 18, batch, maxp, 2, 64, True, p.block_table, p.ctx_len)
        chunk = plan_both(o, p, [20, 30, 15], rows, ws)
        hole = g.choice(65, 12, replace=False)
        chunk.slot[torch.from_numpy(hole)] = -1
        flags = 0
        if trial % 3 == 1:
            chunk.slot[int(hole[0])] = 18 * 16 + 3
            chunk.pos[int(hole[1])] = -1
            flags = BAD_INDEX
        if trial % 3 == 2:
            chunk.seq[int(hole[0])], chunk.slot[int(hole[0])] = 5, 7
            chunk.slot[int(hole[2])] = -9
            flags = BAD_INDEX
        x = bf16(g, rows, 8, 64)
        append_both(kv, rope, x[:, :4], x[:, 4:6], x[:, 6:], chunk, batch, flags)


def test_keys_that_are_no_numbers_fold_as_ever():
    g = np.random.default_rng(19)
    o, p = both_pools(8, 2, 4)
    ws = se.workspace(se.se_page_pool_workspace(2))
    rope = make(g, 64, 128, 0, (0, 0))
    kv = cache(g, 8, 2, 4, 1, 128, True, p.block_table, p.ctx_len)
    chunk = plan_both(o, p, [20, 1], 21, ws)
    x = bf16(g, 21, 3, 128)
    x[4, 1, 5] = math.nan
    x[20, 1] = math.nan
    two = copy_of(kv)
    se.se_rope_append_chunk(kv, rope, None, x[:, 1:2], x[:, 2:], None, chunk, 2, small_ws())
    k2 = x[:, 1:2].clone()
    se.se_qk_rope(rope, chunk.pos, None, k2, None, k2, small_ws())
    se.se_kv_append_chunk(two, k2, x[:, 2:].contiguous(), chunk, 2, small_ws())
    same = lambda a, b: ((a == b) | (a.isnan() & b.isnan())).all()              # noqa: E731
    assert same(kv.k, two.k) and same(kv.meta, two.meta)
    assert not kv.meta[0, 0].isnan().any() and kv.meta[1, 0].isnan().any()


def test_replayed_from_a_graph_and_on_another_stream():
    g = np.random.default_rng(20)
    o, p = both_pools(64, 4, 8)
    ws, small = se.workspace(se.se_page_pool_workspace(4)), small_ws()
    rope = make(g, 128, 128, 0, (1, 1))
    kv = cache(g, 64, 4, 8, 2, 128, True, p.block_table, p.ctx_len)
    chunk = plan_both(o, p, [9, 16, 1, 30], 56, ws)
    x = bf16(g, 56, 8, 128)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    want, start = copy_of(kv), copy_of(kv)
    qw = append_both(want, rope, q, k, v, chunk, 4)
    qo, ko, kw = marked(56, 4, 128), marked(56, 2, 128), marked(56, 2, 128)
    se.se_qk_rope(rope, chunk.pos, None, k, None, kw, small)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        se.se_rope_append_chunk(kv, rope, q, k, v, qo, chunk, 4, small)
        se.se_qk_rope(rope, chunk.pos, None, k, None, ko, small)
    for a, b in ((kv.k, start.k), (kv.v, start.v), (kv.meta, start.meta), (kv.ctx_len, start.ctx_len)):
        a.copy_(b)
    graph.replay()
    assert kv.k.equal(want.k) and kv.meta.equal(want.meta) and kv.ctx_len.equal(want.ctx_len)
    assert qo.equal(qw) and ko.equal(kw)
    # new values in the same buffers
    x.mul_(-0.5)
    qw = append_both(copy_of(start), rope, q, k, v, chunk, 4)
    graph.replay()
    assert qo.equal(qw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = marked(56, 4, 128)
    se.se_rope_append_chunk(copy_of(start), rope, q, k, v, out, chunk, 4, small, stream=side)
    side.synchronize()
    assert out.equal(qw)
