"""GPU parity of the chunk operators (page tables, append, attention) against
the oracle: integers and copied rows exactly, attention within bounds derived
from the roundings it makes."""
import math

import numpy as np
import pytest
import torch

import oracle
from kv_cache_decode_quest_gb300 import binding as se
from kv_cache_decode_quest_gb300 import synth
from oracle import chunk as oc

pytestmark = pytest.mark.gpu
PAGE = 16
BAD_INDEX, CAPACITY, BAD_LENGTH = 1, 2, 4


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def both_pools(num_pages, batch, maxp):
    return oc.Pool(num_pages, batch, maxp), se.PagePool.empty(batch, num_pages, maxp)


def same_pool(o, g):
    n = int(g.n_free)
    assert n == len(o.free) and g.free_pages[:n].cpu().tolist() == o.free
    assert g.n_pages.cpu().tolist() == o.n_pages.tolist()
    assert g.ctx_len.cpu().tolist() == o.ctx.tolist()
    bt = g.block_table.cpu().numpy()
    for b in range(len(o.n_pages)):
        k = o.n_pages[b]
        assert np.array_equal(bt[b, :k], o.block_table[b, :k]), b


def plan_both(o, g, new, rows, ws, chunk=None):
    chunk = chunk or se.Chunk.empty(len(new), rows)
    se.se_chunk_plan(g, i32(new), len(new), chunk, ws)
    start, seq, pos, slot, flags = oc.plan(o, new, rows)
    for name, want in (("start", start), ("seq", seq), ("pos", pos), ("slot", slot)):
        assert np.array_equal(getattr(chunk, name).cpu().numpy(), want), name
    assert se.status_word(ws) == flags
    ws[:4] = 0
    same_pool(o, g)
    return chunk


@pytest.mark.parametrize("batch,hi,pages,maxp", [
    (1, 1, 1, 1), (1, 300, 40, 30), (3, 16, 6, 4), (5, 17, 100, 2), (256, 40, 300, 9),
    (257, 40, 2000, 9), (1025, 33, 900, 5), (2100, 3, 5000, 40)])
def test_plan_and_release_over_many_steps(batch, hi, pages, maxp):
    """Steps of a serving batch with requests that do not fit, that need nothing, that
    finish; every table equal to the oracle's after each."""
    g = np.random.default_rng([5, batch, hi])
    o, p = both_pools(pages, batch, maxp)
    ws = se.workspace(se.se_page_pool_workspace(batch))
    for step in range(6):
        new = g.integers(0, hi + 1, batch)
        new[g.random(batch) < 0.3] = 1
        rows = int(new.sum()) + (0, 7, 1)[step % 3]
        chunk = plan_both(o, p, new, rows, ws)
        plan_both(o, p, new, rows, ws)                       # again: nothing more is taken
        slot, pos, seq = (x.cpu().numpy() for x in (chunk.slot, chunk.pos, chunk.seq))
        for b in range(batch):                                # commit what was served
            mine = pos[seq == b]
            if len(mine) and mine[-1] >= 0:
                o.ctx[b] = mine[-1] + 1
        p.ctx_len.copy_(i32(o.ctx))
        assert len(set(slot[slot >= 0])) == (slot >= 0).sum()
        done = g.random(batch) < 0.3
        se.se_pages_release(p, i32(done), batch, ws)
        oc.release(o, done)
        assert se.status_word(ws) == 0
        same_pool(o, p)


def test_plan_rows_past_max_tokens_take_nothing():
    o, p = both_pools(64, 4, 8)
    ws = se.workspace(se.se_page_pool_workspace(4))
    chunk = plan_both(o, p, [20, 20, 20, 0], 45, ws)
    assert p.n_pages.tolist() == [2, 2, 0, 0]
    assert chunk.slot[40:].tolist() == [-1] * 5 and chunk.seq[40:].tolist() == [2] * 5
    plan_both(o, p, [20, 20, 20, 1], 0, ws)                  # no room for any row


def test_plan_of_nothing():
    p = se.PagePool.empty(2, 4, 4)
    ws = se.workspace(se.se_page_pool_workspace(0))
    chunk = se.Chunk.empty(0, 5)
    chunk.slot.fill_(9)
    se.se_chunk_plan(p, i32([]), 0, chunk, ws)
    assert se.status_word(ws) == 0 and chunk.start.tolist() == [0]
    assert chunk.slot.tolist() == [-1] * 5 and int(p.n_free) == 4


def test_plan_bad_lengths_and_pages():
    o, p = both_pools(16, 5, 4)
    o.ctx[:] = [17, 0, -1, 65, 5]
    o.n_pages[:] = [1, 0, 0, 4, 5]                           # too few, -, -, -, too many
    p.ctx_len.copy_(i32(o.ctx))
    p.n_pages.copy_(i32(o.n_pages))
    ws = se.workspace(se.se_page_pool_workspace(5))
    chunk = se.Chunk.empty(5, 16)
    se.se_chunk_plan(p, i32([3, -2, 1, 1, 1]), 5, chunk, ws)
    assert se.status_word(ws) == BAD_LENGTH
    assert chunk.start.tolist() == [0, 3, 3, 4, 5, 6]
    assert chunk.slot.tolist() == [-1] * 16 and int(p.n_free) == 16
    assert p.n_pages.tolist() == [1, 0, 0, 4, 5]
    # a page outside the cache on the stack, and in the table
    p = se.PagePool.empty(2, 8, 4)
    p.free_pages[7] = 8
    p.free_pages[6] = -3
    ws = se.workspace(se.se_page_pool_workspace(2))
    chunk = se.Chunk.empty(2, 40)
    se.se_chunk_plan(p, i32([33, 2]), 2, chunk, ws)
    assert se.status_word(ws) == BAD_INDEX
    slot = chunk.slot.tolist()
    assert slot[:32] == [-1] * 32 and slot[32] == 2 * 16 and slot[33:35] == [48, 49]
    assert p.block_table[0].tolist() == [-1, -1, 2, -1]


def test_release_of_pages_twice_is_refused():
    p = se.PagePool.empty(2, 4, 4)
    ws = se.workspace(se.se_page_pool_workspace(2))
    p.n_pages.copy_(i32([3, 2]))
    p.block_table[:] = 1
    se.se_pages_release(p, i32([1, 1]), 2, ws)
    assert se.status_word(ws) == CAPACITY
    assert int(p.n_free) == 4 and p.n_pages.tolist() == [3, 2]
    assert p.free_pages.tolist() == [3, 2, 1, 0]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def normal(g, *shape):
    return oracle.widen(synth.f32_to_bf16_bits(g.standard_normal(shape).astype(np.float32)))


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().bfloat16()


def f64(t):
    return t.double().cpu().numpy()


class Cache:
    """A pool and one layer's paged cache on both sides."""

    def __init__(self, g, batch, H, D, maxp, num_pages, summaries=True):
        self.g, self.B, self.H, self.D = g, batch, H, D
        self.o, self.pool = both_pools(num_pages, batch, maxp)
        order = g.permutation(num_pages)
        self.o.free = order.tolist()
        self.pool.free_pages.copy_(i32(order))
        # what no token wrote must never be read as a number
        k = np.full((num_pages, H, PAGE, D), np.nan, dtype=np.float32)
        self.k, self.v = k.astype(np.float64), k.astype(np.float64)
        self.meta = np.zeros((batch, maxp, H, 2, D)) if summaries else None
        self.kv = se.PagedKV(bf16(k), bf16(k), bf16(self.meta) if summaries else None,
                             self.pool.block_table, self.pool.ctx_len)
        self.ws_pool = se.workspace(se.se_page_pool_workspace(batch))
        self.ws = se.workspace(se.se_small_workspace())

    def add(self, new, pad=0, packed=False):
        """Plan and append `new` tokens per sequence; returns the chunk."""
        rows = int(sum(new)) + pad
        chunk = plan_both(self.o, self.pool, new, rows, self.ws_pool)
        wide = normal(self.g, rows, 2 * self.H + 3, self.D)
        kn, vn = wide[:, 1:1 + self.H], wide[:, 1 + self.H:1 + 2 * self.H]
        if packed:
            w = bf16(wide)
            kt, vt = w[:, 1:1 + self.H], w[:, 1 + self.H:1 + 2 * self.H]
        else:
            kt, vt = bf16(kn), bf16(vn)
        se.se_kv_append_chunk(self.kv, kt, vt, chunk, self.B, self.ws)
        oc.append(self.o, self.k, self.v, self.meta, kn, vn,
                  *(getattr(chunk, x).cpu().numpy() for x in ("start", "seq", "pos", "slot")))
        assert se.status_word(self.ws) == 0
        return chunk

    def check(self):
        assert np.array_equal(f64(self.kv.k), self.k, equal_nan=True)
        assert np.array_equal(f64(self.kv.v), self.v, equal_nan=True)
        if self.meta is not None:
            got = f64(self.kv.meta)
            for b in range(self.B):
                n = -(-int(self.o.ctx[b]) // PAGE)
                assert np.array_equal(got[b, :n], self.meta[b, :n]), b
        assert self.pool.ctx_len.tolist() == self.o.ctx.tolist()

    def seq(self, b, h):
        L = int(self.o.ctx[b])
        pages = self.o.block_table[b, :-(-L // PAGE)]
        return (x[pages, h].reshape(-1, self.D)[:L] for x in (self.k, self.v))


@pytest.mark.parametrize("H,D,summaries,packed", [
    (1, 64, True, False), (4, 128, True, True), (8, 64, False, True), (3, 128, True, False)])
def test_append_is_the_oracles(H, D, summaries, packed):
    g = np.random.default_rng([7, H, D])
    c = Cache(g, 6, H, D, 12, 70, summaries)
    for new in ([1, 15, 16, 17, 0, 90], [1, 1, 1, 1, 1, 1], [30, 0, 15, 14, 33, 6],
                [16, 16, 16, 16, 16, 16]):
        c.add(new, pad=len(new) % 4, packed=packed)
        c.check()


def test_append_many_rows_and_few_heads():
    c = Cache(np.random.default_rng(8), 3, 2, 128, 400, 900)
    c.add([5000, 1, 4097])
    c.check()
    c.add([3, 2000, 700], pad=5)
    c.check()


def test_append_chunk_of_one_is_se_kv_append():
    g = np.random.default_rng(9)
    c = Cache(g, 5, 4, 128, 6, 30)
    c.add([15, 16, 1, 47, 0])
    other = se.PagedKV(c.kv.k.clone(), c.kv.v.clone(), c.kv.meta.clone(), c.kv.block_table,
                       c.kv.ctx_len.clone())
    chunk = plan_both(c.o, c.pool, [1] * 5, 5, c.ws_pool)
    k, v = bf16(normal(g, 5, 4, 128)), bf16(normal(g, 5, 4, 128))
    se.se_kv_append(other, k, v, 5, c.ws)
    se.se_kv_append_chunk(c.kv, k, v, chunk, 5, c.ws)
    for x in ("k", "v", "meta", "ctx_len"):
        assert torch.equal(torch.nan_to_num(getattr(c.kv, x)), torch.nan_to_num(getattr(other, x))), x


def test_append_drops_what_has_no_page():
    c = Cache(np.random.default_rng(10), 3, 2, 64, 4, 5)
    c.o.free = c.o.free[-2:]
    c.pool.free_pages[:2] = i32(c.o.free)
    c.pool.n_free.fill_(2)
    c.add([16, 40, 3])                       # the second and third find no page
    c.check()
    assert c.pool.ctx_len.tolist() == [16, 0, 0]
    before = c.kv.k.clone()
    bad = se.Chunk(i32([0, 1, 2, 3]), i32([0, 3, 0]), i32([0, 0, 64]), i32([80, 0, 0]))
    k = bf16(normal(c.g, 3, 2, 64))
    se.se_kv_append_chunk(c.kv, k, k, bad, 3, c.ws)
    assert se.status_word(c.ws) == BAD_INDEX
    assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(c.kv.k))
    assert c.pool.ctx_len.tolist() == [16, 0, 0]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def bounds(q, k, v, pos0, scale, window, sink, out_f32, absent=()):
    """(out, lse, bound of out, bound of lse) of rows q [n][G][D].

    A logit is a sum of D exact products in fp32 in steps of 16 (each rounded by at most
    2^-23 of the sum of magnitudes s), then scaled and shifted (three more such
    roundings), and its exponential has a relative error of 2^-22: d = 2^-22 +
    (D/16 + 3) 2^-23 s bounds each weight's relative error, and twice that the normalised
    one's.  A weight is rounded to bf16 (2^-8) or to two bf16 terms (2^-16)
    before the product with v, whose fp32 sums over at most L/16 steps round by
    2^-23 of the sum of magnitudes a = sum p |v| each; the result is rounded to its type."""
    out, lse = oracle.chunk_attend(q, k, v, pos0, scale, window, sink, absent)
    a, _ = oracle.chunk_attend(q, k, np.abs(v), pos0, scale, window, sink, absent)
    D, L = q.shape[-1], max(1, len(k))
    s = abs(scale) * np.abs(q).sum(-1).max() * max(1e-30, np.abs(k).max()) if len(k) else 0.0
    s = min(s, abs(scale) * float((np.abs(q).reshape(-1, D) @ np.abs(k).T).max())) if len(k) else 0.0
    d = 2.0 ** -22 + (D / 16 + 3) * 2.0 ** -23 * s
    p = 2.0 ** -16 if out_f32 else 2.0 ** -8
    rnd = 2.0 ** -24 if out_f32 else 2.0 ** -8
    tol = a * (p + 2 * d + (L / 16 + 8) * 2.0 ** -23) * 1.01 + np.abs(out) * rnd + 1e-30
    ltol = d + 2.0 ** -22 * (2 + np.abs(np.where(np.isinf(lse), 0, lse)))
    return out, lse, tol, ltol


class Attn:
    def __init__(self, cache, G, out_f32=False, scale=None, window=0, sink=0, packed=False):
        self.c, self.G, self.f32 = cache, G, out_f32
        self.Hq = cache.H * G
        self.scale = 1.0 / math.sqrt(cache.D) if scale is None else scale
        self.window, self.sink, self.packed = window, sink, packed
        self.ws = None

    def run(self, chunk, stream=None):
        c = self.c
        rows = chunk.seq.numel()
        wide = normal(c.g, rows, self.Hq + 2, c.D)
        self.q = wide[:, 1:1 + self.Hq]
        w = bf16(wide)
        self.qt = w[:, 1:1 + self.Hq] if self.packed else w[:, 1:1 + self.Hq].contiguous()
        self.out = torch.full((rows, self.Hq, c.D), 7.0, device="cuda",
                              dtype=torch.float32 if self.f32 else torch.bfloat16)
        self.lse = torch.full((rows, self.Hq), 7.0, device="cuda")
        if self.ws is None:
            self.ws = se.workspace(se.se_chunk_attn_workspace(c.B, rows, c.H, self.Hq, c.D))
        self.call(chunk, stream)

    def call(self, chunk, stream=None):
        c = self.c
        se.se_chunk_attn(c.kv, self.qt, chunk, c.B, self.Hq, self.scale, self.out, self.lse,
                         self.ws, out_dtype=int(self.f32), window=self.window, sink=self.sink,
                         stream=stream)

    def check(self, chunk, status=0, rows=None, absent=None):
        c, G = self.c, self.G
        assert se.status_word(self.ws) == status
        out, lse = f64(self.out), f64(self.lse)
        start, pos = chunk.start.tolist(), chunk.pos.cpu().numpy()
        for b in range(c.B):
            s0, s1 = start[b], start[b + 1]
            if s0 == s1:
                continue
            pick = range(s0, s1) if rows is None or s1 - s0 <= rows else \
                sorted(set(np.linspace(s0, s1 - 1, rows).astype(int)))
            for h in range(c.H):
                k, v = c.seq(b, h)
                gone = [] if absent is None else absent.get(b, [])
                # runs of consecutive picked rows
                pick = list(pick)
                runs = np.split(pick, 1 + np.flatnonzero(np.diff(pick) != 1))
                for r in runs:
                    a, z = int(r[0]), int(r[-1]) + 1
                    want, wl, tol, ltol = bounds(self.q[a:z, h * G:(h + 1) * G], k, v, int(pos[a]),
                                                 self.scale, self.window, self.sink, self.f32, gone)
                    got, gl = out[a:z, h * G:(h + 1) * G], lse[a:z, h * G:(h + 1) * G]
                    err = np.abs(got - want)
                    assert np.all(err <= tol), (b, h, a, float((err - tol).max()))
                    assert np.array_equal(np.isneginf(gl), np.isneginf(wl)), (b, h, a)
                    fin = np.isfinite(wl)
                    assert np.all(np.abs(gl[fin] - wl[fin]) <= ltol[fin]), (b, h, a)
        assert np.all(out[start[c.B]:] == 7.0) and np.all(lse[start[c.B]:] == 7.0)


def held(g, B, H, D, ctx, extra, summaries=False):
    maxp = max(-(-(c + n) // PAGE) for c, n in zip(ctx, extra)) + 1
    pages = sum(-(-(c + n) // PAGE) for c, n in zip(ctx, extra)) + 2
    c = Cache(g, B, H, D, maxp, pages, summaries)
    if any(ctx):
        c.add(ctx)
    return c


# (H, G, D, ctx, new): one token to long ones, odd sizes, groups, empty sequences,
# lengths on both sides of pages, 128-key tiles and row blocks
SHAPES = [
    (1, 1, 64, [0], [1]), (1, 4, 64, [2047], [1]), (2, 8, 128, [0, 5, 0], [1, 0, 16]),
    (4, 8, 128, [127, 128, 129, 0], [1, 1, 1, 128]), (2, 2, 128, [15, 16, 17], [1, 130, 63]),
    (1, 16, 128, [100, 0], [17, 40]), (2, 1, 64, [300, 3], [257, 129]),
    (1, 4, 128, [0], [513]), (2, 16, 64, [255, 640], [1, 2]), (1, 8, 64, [1000, 31], [33, 65]),
    (3, 2, 64, [77, 500, 0, 1], [5, 128, 9, 300]),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("H,G,D,ctx,new", SHAPES)
def test_attention_is_the_oracles(H, G, D, ctx, new, f32):
    g = np.random.default_rng([12, H, G, D, len(ctx)])
    c = held(g, len(ctx), H, D, ctx, new)
    chunk = c.add(new, pad=3)
    a = Attn(c, G, f32, packed=len(ctx) % 2 == 1)
    a.run(chunk)
    a.check(chunk, rows=48)


@pytest.mark.parametrize("window,sink", [(1, 0), (16, 0), (100, 4), (129, 130), (1000, 17)])
@pytest.mark.parametrize("G,D", [(1, 64), (8, 128)])
def test_window_and_sink(G, D, window, sink):
    g = np.random.default_rng([13, G, window])
    ctx, new = [0, 700, 1], [200, 40, 1]
    c = held(g, 3, 2, D, ctx, new)
    chunk = c.add(new)
    for f32 in (False, True):
        a = Attn(c, G, f32, window=window, sink=sink)
        a.run(chunk)
        a.check(chunk, rows=40)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3, 4.0])
def test_scales(scale):
    g = np.random.default_rng([14])
    c = held(g, 2, 1, 128, [90, 0], [30, 70])
    chunk = c.add([30, 70])
    a = Attn(c, 4, True, scale=scale)
    a.run(chunk)
    a.check(chunk, rows=30)


def test_long_context_split_over_the_gpu():
    g = np.random.default_rng([15])
    for D, G in ((128, 8), (64, 4)):
        c = held(g, 2, 1, D, [20000, 9001], [3, 1])
        chunk = c.add([3, 1])
        for f32 in (False, True):
            a = Attn(c, G, f32)
            a.run(chunk)
            a.check(chunk)


@pytest.mark.parametrize("H,G,D,ctx,new", [
    (1, 8, 128, [9000], [64]), (1, 1, 64, [7003], [300]), (1, 16, 128, [6000, 5000], [17, 3])])
def test_blocks_cut_into_many_pieces(H, G, D, ctx, new):
    """Few blocks over many keys: every SM takes a part, joined in two levels."""
    g = np.random.default_rng([22, G])
    c = held(g, len(ctx), H, D, ctx, new)
    chunk = c.add(new)
    for f32 in (False, True):
        a = Attn(c, G, f32)
        a.run(chunk)
        a.check(chunk, rows=10)
        first = a.out.clone()
        a.call(chunk)
        assert torch.equal(first, a.out)


def test_many_sequences():
    """More sequences than threads of a block: single tokens, empty ones, a few chunks."""
    g = np.random.default_rng([23])
    B = 900
    ctx = g.integers(0, 60, B)
    new = g.integers(0, 3, B)
    new[[3, 400, 899]] = [70, 33, 17]
    c = Cache(g, B, 1, 64, 10, int(sum(-(-(a + b) // PAGE) for a, b in zip(ctx, new))) + 1, False)
    c.add(list(ctx))
    chunk = c.add(list(new), pad=1)
    a = Attn(c, 4)
    a.run(chunk)
    a.check(chunk, rows=8)
    # the same rows in packed arrays with room for many more
    wide = se.Chunk.empty(B, 60000)
    wide.start.copy_(chunk.start)
    for x in ("seq", "pos", "slot"):
        getattr(wide, x)[:len(chunk.seq)] = getattr(chunk, x)
    out, lse = a.out.clone(), a.lse.clone()
    a.qt = torch.cat([a.qt, torch.zeros(60000 - len(a.qt), 4, 64, dtype=a.qt.dtype, device="cuda")])
    a.out = torch.full((60000, 4, 64), 7.0, dtype=out.dtype, device="cuda")
    a.lse = torch.full((60000, 4), 7.0, device="cuda")
    a.ws = se.workspace(se.se_chunk_attn_workspace(B, 60000, 1, 4, 64))
    a.call(wide)
    assert torch.equal(a.out[:len(out)], out) and torch.equal(a.lse[:len(lse)], lse)
    assert torch.all(a.out[len(out):] == 7.0) and torch.all(a.lse[len(out):] == 7.0)


def test_rows_before_the_end_of_what_is_held():
    """Positions in the middle of a longer history (the later keys are not seen)."""
    g = np.random.default_rng([24])
    c = held(g, 2, 2, 128, [500, 77], [1, 1])
    chunk = c.add([1, 1])
    n = [150, 20]
    pos0 = [33, 50]
    seq = np.repeat([0, 1], n)
    pos = np.concatenate([p + np.arange(k) for p, k in zip(pos0, n)])
    mid = se.Chunk(i32([0, 150, 170]), i32(seq), i32(pos), i32(np.zeros(170)))
    for window in (0, 40):
        a = Attn(c, 4, window=window)
        a.run(mid)
        a.check(mid, rows=30)


def test_longest_window_and_sink():
    """Window and sink of 2^31 - 1, alone and together, see what no window does."""
    g = np.random.default_rng([25])
    c = held(g, 2, 2, 64, [700, 0], [40, 130])
    chunk = c.add([40, 130])
    a = Attn(c, 4)
    a.run(chunk)
    a.check(chunk, rows=20)
    out, lse = a.out.clone(), a.lse.clone()
    for a.window, a.sink in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        a.out.fill_(7.0)
        a.lse.fill_(7.0)
        a.call(chunk)
        assert se.status_word(a.ws) == 0
        assert torch.equal(a.out, out) and torch.equal(a.lse, lse), (a.window, a.sink)


def test_growing_maximum():
    """Keys whose logits grow along the sequence: every tile raises the running maximum."""
    g = np.random.default_rng([16])
    c = Cache(g, 1, 1, 128, 130, 130)
    n = 2000
    q = normal(g, 1, 2, 128)[0]
    k = np.outer(np.linspace(-40, 40, n), np.sign(q[0])) / 8
    k = oracle.widen(synth.f32_to_bf16_bits(k.astype(np.float32)))[:, None]
    v = normal(g, n, 1, 128)
    chunk = plan_both(c.o, c.pool, [n], n, c.ws_pool)
    se.se_kv_append_chunk(c.kv, bf16(k), bf16(v), chunk, 1, c.ws)
    oc.append(c.o, c.k, c.v, c.meta, k, v,
              *(getattr(chunk, x).cpu().numpy() for x in ("start", "seq", "pos", "slot")))
    for f32 in (False, True):
        a = Attn(c, 2, f32)
        a.run(chunk)
        a.q = np.broadcast_to(q, a.q.shape)
        a.qt = bf16(a.q)
        a.call(chunk)
        a.check(chunk, rows=12)


@pytest.mark.parametrize("jump", [20.0, 150.0, 3000.0])
def test_sudden_jumps(jump):
    """Single keys whose logits lie far above all before them, at the borders of tiles and
    inside; behind the last one everything else vanishes."""
    g = np.random.default_rng([25])
    n, D = 700, 64
    c = Cache(g, 1, 1, D, 45, 45)
    q = np.ones((n, 2, D))
    k = normal(g, n, 1, D) / 8
    for i, at in enumerate((1, 127, 128, 200, 383, 511, 640)):
        k[at] = oracle.widen(synth.f32_to_bf16_bits(np.full((1, D), (i + 1) * jump / 8, np.float32)))
    v = normal(g, n, 1, D)
    chunk = plan_both(c.o, c.pool, [n], n, c.ws_pool)
    se.se_kv_append_chunk(c.kv, bf16(k), bf16(v), chunk, 1, c.ws)
    oc.append(c.o, c.k, c.v, c.meta, k, v,
              *(getattr(chunk, x).cpu().numpy() for x in ("start", "seq", "pos", "slot")))
    for f32 in (False, True):
        a = Attn(c, 2, f32)
        a.run(chunk)
        a.q, a.qt = q, bf16(q)
        a.call(chunk)
        a.check(chunk, rows=16)


def test_refused_rows_and_missing_pages():
    g = np.random.default_rng([17])
    c = held(g, 3, 2, 128, [40, 0, 300], [5, 20, 5])
    c.o.free = c.o.free[-1:]
    c.pool.free_pages[:1] = i32(c.o.free)
    c.pool.n_free.fill_(1)
    # the second needs two pages and one is left; the third needs one (305 tokens, 19
    # pages held) and does not overtake
    chunk = c.add([5, 20, 5])
    assert chunk.pos[5:].tolist() == [-1] * 25
    a = Attn(c, 4)
    a.run(chunk)
    a.check(chunk)
    assert torch.all(a.out[5:] == 0) and torch.all(torch.isneginf(a.lse[5:]))
    # pages of keys that refused rows do not see are not looked up
    c.pool.block_table[2, 3] = c.kv.k.shape[0]
    a.run(chunk)
    a.check(chunk)


@pytest.mark.parametrize("f32", [False, True])
def test_missing_pages_count_as_absent(f32):
    g = np.random.default_rng([21])
    c = held(g, 2, 2, 128, [140, 300], [5, 40])
    chunk = c.add([5, 40])
    c.pool.block_table[0, 0] = -1
    c.pool.block_table[1, 3] = c.kv.k.shape[0]
    c.pool.block_table[1, 11] = -7
    a = Attn(c, 4, f32)
    a.run(chunk)
    a.check(chunk, status=BAD_INDEX,
            absent={0: [*range(16)], 1: [*range(48, 64), *range(176, 192)]})


def test_lengths_that_do_not_fit():
    g = np.random.default_rng([18])
    c = held(g, 2, 1, 64, [40, 40], [8, 8])
    chunk = c.add([8, 8])
    a = Attn(c, 2)
    # fewer tokens held than the rows' positions say: the rows see what is held
    c.o.ctx[1] = 45
    c.pool.ctx_len[1] = 45
    a.run(chunk)
    a.check(chunk, status=BAD_LENGTH)
    # starts past the rows and descending
    a.ws[:4] = 0
    a.out.fill_(7)
    odd = se.Chunk(i32([0, 99, 8]), chunk.seq, chunk.pos, chunk.slot)
    a.call(odd)
    assert se.status_word(a.ws) == BAD_LENGTH
    a.ws[:4] = 0
    a.call(chunk)
    a.check(chunk, status=BAD_LENGTH)


def test_same_result_every_time_on_streams_and_in_graphs():
    g = np.random.default_rng([19])
    ctx, new = [3000, 50, 0, 777], [40, 1, 150, 1]
    c = held(g, 4, 2, 128, ctx, new)
    chunk = c.add(new, pad=2)
    a = Attn(c, 8)
    a.run(chunk)
    a.check(chunk, rows=24)
    first = (a.out.clone(), a.lse.clone())
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.out.fill_(7)
        torch.cuda.synchronize()
        a.call(chunk, stream=other)
        other.synchronize()
        assert torch.equal(a.out, first[0]) and torch.equal(a.lse, first[1])
    # a captured step: plan, append and attention, replayed with other lengths
    new_len = i32(new)
    k, v = (bf16(normal(g, 194, 2, 128)) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        se.se_chunk_plan(c.pool, new_len, 4, chunk, c.ws_pool)
        se.se_kv_append_chunk(c.kv, k, v, chunk, 4, c.ws)
        a.call(chunk)
    torch.cuda.synchronize()
    for nxt in ([0, 5, 1, 2], [1, 0, 0, 1]):
        new_len.copy_(i32(nxt))
        a.out.fill_(7)
        a.lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want = oc.plan(c.o, nxt, 194)
        assert np.array_equal(chunk.slot.cpu().numpy(), want[3])
        oc.append(c.o, c.k, c.v, None, f64(k), f64(v), *want[:4])
        a.check(chunk, rows=24)


def test_one_workspace_for_calls_of_any_shape():
    g = np.random.default_rng([20])
    shapes = [([900], [1]), ([10, 2000], [300, 3]), ([0], [700]), ([900], [1])]
    size = max(se.se_chunk_attn_workspace(len(c), sum(n) + 1, 1, 8, 64) for c, n in shapes)
    ws = se.workspace(size)
    for ctx, new in shapes:
        c = held(g, len(ctx), 1, 64, ctx, new)
        chunk = c.add(new, pad=1)
        a = Attn(c, 8)
        a.ws = ws
        a.run(chunk)
        a.check(chunk, rows=24)
