"""GPU: the calls of a step with drafted tokens together (page tables, rotation and append, attention,
verification, truncation), with forked samples, against a plain record of what every sequence holds."""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_decode_quest_gb300 import binding as se
from kv_cache_decode_quest_gb300.workloads import DraftRun
from tests.parity import TOL_BF16, TOL_F32, max_abs
from tests.test_gpu_chunk import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


class Record:
    """Each sequence's rotated keys and its values, layer by layer, as lists of rows."""

    def __init__(self, run):
        self.run = run
        self.k = [[[] for _ in run.kv] for _ in range(run.B)]
        self.v = [[[] for _ in run.kv] for _ in range(run.B)]

    def append(self, qkv, new):
        """The rows as the library rotates them alone; queries returned."""
        run, q = self.run, []
        for layer, (x, rope) in enumerate(zip(qkv, run.ropes)):
            Hq, H = run.Hq, run.H
            pos = run.chunk.pos
            qr, kr = torch.zeros_like(x[:, :Hq]), torch.zeros_like(x[:, Hq:Hq + H])
            se.se_qk_rope(rope, pos, x[:, :Hq], x[:, Hq:Hq + H], qr, kr, run.ws_small)
            q.append(qr.double().cpu().numpy())
            k, v = kr.double().cpu().numpy(), x[:, Hq + H:].double().cpu().numpy()
            at = 0
            for b, n in enumerate(new):
                self.k[b][layer] += list(k[at:at + n])
                self.v[b][layer] += list(v[at:at + n])
                at += n
        return q

    def cut(self, b, n):
        for x in (self.k, self.v):
            x[b] = [rows[:n] for rows in x[b]]

    def fork(self, b, src):
        for x in (self.k, self.v):
            x[b] = [list(rows) for rows in x[src]]

    def same_caches(self):
        run = self.run
        for b in range(run.B):
            L = len(self.k[b][0])
            assert int(run.pool.ctx_len[b]) == L
            bt = run.pool.block_table[b, :-(-L // 16)].long()
            for layer, kv in enumerate(run.kv):
                for x, want in ((kv.k, self.k), (kv.v, self.v)):
                    got = x[bt].transpose(0, 1).reshape(run.H, -1, run.D)[:, :L]
                    if L:
                        assert np.array_equal(got.double().cpu().numpy(),
                                              np.array(want[b][layer]).transpose(1, 0, 2))
                for p in range(-(-L // 16)):
                    rows = np.array(self.k[b][layer][16 * p:16 * p + 16])
                    got = kv.meta[b, p].double().cpu().numpy()
                    assert np.array_equal(got[:, 0], rows.min(0)) and np.array_equal(got[:, 1], rows.max(0))

    def attention(self, q, new, tol):
        run, G = self.run, self.run.Hq // self.run.H
        for layer in range(len(run.kv)):
            out, at = run.out[layer].double().cpu().numpy(), 0
            for b, n in enumerate(new):
                L = len(self.k[b][layer])
                for h in range(run.H) if n else ():
                    K, V = (np.array(x[b][layer])[:, h] for x in (self.k, self.v))
                    for i in {0, n - 1}:
                        o, _ = oracle.chunk_attend(q[layer][at + i:at + i + 1, h * G:(h + 1) * G], K, V,
                                                   L - n + i, run.scale)
                        assert max_abs(out[at + i, h * G:(h + 1) * G], o[0]) <= tol
                at += n


@pytest.mark.parametrize("D,G,H,vocab,drafter,out_dtype", [
    (128, 8, 2, 300, True, 0), (64, 4, 1, 5001, True, 1), (64, 1, 4, 77, False, 0)])
def test_steps_with_drafts_and_samples(D, G, H, vocab, drafter, out_dtype):
    """Three prompts, samples forked from them, five steps of drafts of which some stay: caches, summaries,
    attention and accepted tokens equal what a plain record gives, no page is lost."""
    g = np.random.default_rng([41, D, G, vocab])
    B, rows = 7, 7 * 60
    w = [torch.from_numpy(1 + 0.2 * g.standard_normal(D)).bfloat16().cuda() for _ in range(2)]
    ropes = [se.Rope.make(D, q_weight=w[0], k_weight=w[1]),
             se.Rope.make(D // 2, base=1e6, scaling=se.SE_ROPE_YARN, factor=4.0, original_len=128.0,
                          layout=se.SE_ROPE_PAIRS)]
    run = DraftRun(B, G * H, H, D, num_pages=90, max_pages=14, max_rows=rows, vocab=vocab, ropes=ropes,
                   out_dtype=out_dtype)
    rec = Record(run)

    def feed(new):
        qkv = [torch.from_numpy(g.standard_normal((rows, (G + 2) * H, D))).bfloat16().cuda()
               for _ in ropes]
        run.feed(qkv, i32(new))
        q = rec.append(qkv, new)
        rec.attention(q, new, TOL_F32 if out_dtype else TOL_BF16)

    feed([50, 33, 16, 0, 0, 0, 0])
    run.fork(i32([-1, -1, -1, 0, 0, 2, 1]))
    for b, src in ((3, 0), (4, 0), (5, 2), (6, 1)):
        rec.fork(b, src)
    rec.same_caches()
    accepted = 0
    for step in range(5):
        new = g.integers(1, 9, B)
        new[step % B] = 20
        before = run.pool.ctx_len.tolist()
        feed(new)
        x = g.standard_normal((rows, vocab)) * 2
        soft = lambda y: torch.softmax(torch.from_numpy(y).float(), 1).cuda()     # noqa: E731
        p, q = soft(x), soft(x + 0.3 * g.standard_normal(x.shape)) if drafter else None
        tok = np.roll(np.where(g.random(rows) < 0.7, x.argmax(1), g.integers(0, vocab, rows)), 1)
        au, su = g.random(rows).astype(np.float32), g.random(B).astype(np.float32)
        run.check(p, q, i32(tok), torch.from_numpy(au).cuda(), torch.from_numpy(su).cuda())
        at, n_accepted = 0, run.n_accepted.tolist()
        pn = p.cpu().numpy()
        qn = None if q is None else q.cpu().numpy()
        for b, n in enumerate(new):
            s = slice(at, at + n)
            want = oracle.draft_verify(pn[s], None if qn is None else qn[s], tok[s], au[s], su[b], before[b])
            assert (n_accepted[b], int(run.next_token[b]), int(run.keep[b])) == want
            rec.cut(b, want[2])
            at += n
        accepted += sum(n_accepted)
        rec.same_caches()
        if step == 2:                                     # samples end, others begin from what stands
            run.cut(i32([-1, 0, -1, -1, 0, -1, -1]))
            run.fork(i32([-1, 3, -1, -1, 3, -1, -1]))
            rec.fork(1, 3)
            rec.fork(4, 3)
            rec.same_caches()
    assert 0 < accepted and run.status() == 0
    assert int(run.refs.max()) >= 1
    run.cut(i32([0] * B))
    assert int(run.pool.n_free) == 90 and not run.refs.any() and run.status() == 0
    assert sorted(run.pool.free_pages.tolist()) == list(range(90))


def test_the_same_steps_captured_in_a_graph():
    """feed and check as one graph with fixed buffers, replayed with new inputs, against the calls."""
    g = np.random.default_rng(42)
    B, rows, vocab, D = 4, 24, 200, 128
    make = lambda: DraftRun(B, 8, 2, D, num_pages=64, max_pages=16, max_rows=rows, vocab=vocab,   # noqa: E731
                            ropes=[se.Rope.make(D)])
    one, two = make(), make()
    qkv = torch.zeros(rows, 12, D, dtype=torch.bfloat16, device="cuda")
    p, q = (torch.zeros(rows, vocab, device="cuda") for _ in range(2))
    au, su, tok, new = torch.zeros(rows, device="cuda"), torch.zeros(B, device="cuda"), i32([0] * rows), i32([6] * B)

    def step(run):
        run.feed([qkv], new)
        run.check(p, q, tok, au, su)
    step(make())                                              # (kernels loaded)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one)
    for _ in range(5):
        qkv.copy_(torch.from_numpy(g.standard_normal(qkv.shape)))
        x = g.standard_normal((rows, vocab)) * 2
        p.copy_(torch.softmax(torch.from_numpy(x).float(), 1))
        q.copy_(torch.softmax(torch.from_numpy(x + 0.3 * g.standard_normal(x.shape)).float(), 1))
        tok.copy_(i32(np.roll(x.argmax(1), 1)))
        au.copy_(torch.from_numpy(g.random(rows)))
        su.copy_(torch.from_numpy(g.random(B)))
        graph.replay()
        step(two)
        for a, b in ((one.keep, two.keep), (one.next_token, two.next_token), (one.kv[0].k, two.kv[0].k),
                     (one.kv[0].meta, two.kv[0].meta), (one.out[0], two.out[0]),
                     (one.pool.block_table, two.pool.block_table), (one.pool.n_free, two.pool.n_free)):
            assert a.equal(b)
    assert one.status() == two.status() == 0


def test_quest_decodes_from_a_forked_cache():
    """A sample forked from a prompt selects and attends as the prompt itself does."""
    g = np.random.default_rng(43)
    D, L = 128, 700
    run = DraftRun(2, 8, 2, D, num_pages=100, max_pages=48, max_rows=L, vocab=10, ropes=[se.Rope.make(D)])
    run.feed([torch.from_numpy(g.standard_normal((L, 12, D))).bfloat16().cuda()], i32([L, 0]))
    run.fork(i32([-1, 0]))
    one = lambda h: torch.from_numpy(g.standard_normal((1, h, D))).bfloat16().cuda().expand(2, h, D).contiguous()  # noqa: E731
    q, k, v = one(8), one(2), one(2)
    rope = run.ropes[0]
    se.se_qk_rope(rope, run.pool.ctx_len, q, k, q, k, run.ws_small)
    units, maxp = 4, 48
    sel = torch.zeros(units, maxp, dtype=torch.int32, device="cuda")
    n_sel, budget = i32([0] * units), i32([160, 160])
    view = se.View.empty(units, maxp)
    out = torch.zeros(2, 8, D, device="cuda")
    ws = se.workspace(se.se_quest_step_workspace(2, 2, 8, D, maxp))
    se.se_quest_step(run.kv[0], k, v, q, 2, 8, budget, run.scale, sel, n_sel, view, out, None, ws, out_dtype=1)
    assert se.status_word(ws) == 0 and run.pool.ctx_len.tolist() == [L + 1, L + 1]
    assert n_sel.tolist() == [10] * 4 and sel[:2].equal(sel[2:])
    assert max_abs(out[0].double().cpu().numpy(), out[1].double().cpu().numpy()) <= TOL_F32
    # the tokens went to pages of their own
    a, b = run.pool.block_table[:, L // 16].tolist()
    assert a != b and run.pool.block_table[0, :L // 16].equal(run.pool.block_table[1, :L // 16])


def test_two_runs_on_two_streams():
    """Steps of two runs in flight at once, each with workspaces of its own: as one after the other."""
    B, rows, vocab, D = 6, 48, 4000, 64
    new, make = i32([8] * B), lambda: DraftRun(B, 4, 2, D, num_pages=200, max_pages=30, max_rows=rows,   # noqa: E731
                                               vocab=vocab, ropes=[se.Rope.make(D), se.Rope.make(32)])
    g = np.random.default_rng(44)
    data = []
    for _ in range(2):
        x = g.standard_normal((rows, vocab)) * 2
        p = torch.softmax(torch.from_numpy(x).float(), 1).cuda()
        qkv = [torch.from_numpy(g.standard_normal((rows, 8, D))).bfloat16().cuda() for _ in range(2)]
        data.append((qkv, p, i32(np.roll(x.argmax(1), 1)), torch.from_numpy(g.random(rows)).float().cuda(),
                     torch.from_numpy(g.random(B)).float().cuda()))

    def step(run, d):
        run.feed(d[0], new)
        run.check(d[1], None, d[2], d[3], d[4])
    alone, both = [make(), make()], [make(), make()]
    for run, d in zip(alone, data):
        for _ in range(6):
            step(run, d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(6):
        for run, d, s in zip(both, data, streams):
            with torch.cuda.stream(s):
                step(run, d)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert a.status() == b.status() == 0
        for x, y in ((a.keep, b.keep), (a.next_token, b.next_token), (a.kv[1].k, b.kv[1].k),
                     (a.kv[0].meta, b.kv[0].meta), (a.pool.free_pages, b.pool.free_pages)):
            assert x.equal(y)
