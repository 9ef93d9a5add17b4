"""GPU parity of the draft verification against the oracle's exact arithmetic: every integer equal."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from oracle import verify as V
from tests.test_gpu_chunk import i32

pytestmark = pytest.mark.gpu
BAD_INDEX, BAD_LENGTH, BAD_VALUE = 1, 4, 16


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


class Case:
    """Rows of some sequences with probabilities, drafts and random numbers."""

    def __init__(self, g, rows, vocab, dtype=torch.float32, drafter=True, pad=0, stride=0, sharp=2.0):
        B, n = len(rows), int(np.sum(rows))
        self.rows, self.vocab, self.g = rows, vocab, g
        x = g.standard_normal((n + pad, vocab)) * sharp
        soft = lambda y: np.exp(y) / np.exp(y).sum(1, keepdims=True)            # noqa: E731
        self.p = self.place(soft(x), dtype, stride)
        q = soft(x + 0.5 * g.standard_normal(x.shape))
        self.q = self.place(q, dtype, stride) if drafter else None
        tok = np.zeros(n + pad, dtype=int)
        for t in range(n + pad - 1):                       # drawn by the drafter, sometimes the target's best
            tok[t + 1] = g.choice(vocab, p=q[t]) if g.random() < 0.8 else x[t].argmax()
        self.tokens = i32(tok)
        self.accept_u = torch.from_numpy(g.random(n + pad).astype(np.float32)).cuda()
        self.sample_u = torch.from_numpy(g.random(B).astype(np.float32)).cuda()
        self.chunk = se.Chunk.empty(B, n + pad)
        start = np.concatenate([[0], np.cumsum(rows)])
        self.chunk.start.copy_(i32(start))
        self.first = g.integers(0, 50000, B)
        for b, r in enumerate(rows):
            self.chunk.pos[start[b]:start[b + 1]] = i32(self.first[b] + np.arange(r))
        self.out = [torch.full((B,), 55, dtype=torch.int32, device="cuda") for _ in range(3)]

    @staticmethod
    def place(x, dtype, stride):
        t = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
        if not stride:
            return t
        wide = torch.full((x.shape[0], stride), float("nan"), dtype=dtype, device="cuda")
        wide[:, :x.shape[1]] = t
        return wide[:, :x.shape[1]]

    def run(self, ws=None, stream=None):
        B = len(self.rows)
        ws = se.workspace(se.se_draft_verify_workspace(B, self.vocab)) if ws is None else ws
        se.se_draft_verify(self.p, self.q, self.tokens, self.accept_u, self.sample_u, self.chunk, B,
                           *self.out, ws, stream=stream)
        return [x.tolist() for x in self.out], se.status_word(ws)

    def want(self):
        p, tok = self.p.float().cpu().numpy(), self.tokens.cpu().numpy()
        q = None if self.q is None else self.q.float().cpu().numpy()
        u, su = self.accept_u.cpu().numpy(), self.sample_u.cpu().numpy()
        got, at = [], 0
        for b, n in enumerate(self.rows):
            if n == 0:
                got.append((0, -1, -1))
                continue
            s = slice(at, at + n)
            a, t, keep = V.verify(p[s], None if q is None else q[s], tok[s], u[s], su[b],
                                  int(self.first[b]))
            got.append((a, -1 if t is None else t, keep))
            at += n
        return [list(x) for x in zip(*got)]


@pytest.mark.parametrize("rows,vocab", [
    ([1], 1), ([2], 1), ([3], 2), ([5], 32), ([1, 1, 1], 7), ([4, 1, 6, 2], 100), ([3] * 20, 1000),
    ([0, 5, 0, 0, 3, 0], 333), ([40], 50), ([34, 70], 11), ([2, 3], 1023), ([2, 3], 1024), ([2, 3], 1025),
    ([3, 2, 4], 5003), ([2] * 300, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
def test_every_shape(rows, vocab, dtype, drafter):
    g = np.random.default_rng([21, len(rows), vocab, drafter])
    # rows one after another (any alignment), rows of a wider array, padded rows
    for stride, pad in ((0, 0), (vocab + 3, 0), (vocab + 8, 5)):
        c = Case(g, rows, vocab, dtype, drafter, pad, stride)
        got, status = c.run()
        assert got == c.want() and status == 0, stride


def test_all_drafts_may_stay():
    g = np.random.default_rng(22)
    c = Case(g, [33, 65, 1, 32], 40)
    c.accept_u.zero_()
    got, _ = c.run()
    assert got == c.want() and got[0] == [32, 64, 0, 31]


def test_large_vocabularies():
    """Many tiles and blocks; the sums in 64 bits (a draw on a border has a chance of 10^-9)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for vocab, B, n, dtype in ((131071, 5, 4, torch.float32), (262147, 2, 3, torch.float32),
                               (200003, 40, 2, torch.bfloat16), (1 << 22, 1, 2, torch.float32)):
        rows = B * n
        p, q = (torch.softmax(3 * torch.randn(rows, vocab, generator=g, device="cuda"), 1).to(dtype)
                for _ in range(2))
        c = Case.__new__(Case)
        c.rows, c.vocab, c.p, c.q = [n] * B, vocab, p, q
        c.tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
        c.accept_u, c.sample_u = (torch.rand(k, generator=g, device="cuda") for k in (rows, B))
        c.accept_u[torch.rand(rows, generator=g, device="cuda") < 0.5] = 0
        c.chunk = se.Chunk.empty(B, rows)
        c.chunk.start.copy_(torch.arange(B + 1, device="cuda") * n)
        c.chunk.pos.copy_(torch.arange(rows, device="cuda"))
        c.out = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3)]
        (stay, token, keep), status = c.run()
        assert status == 0
        for b in range(B):
            t, a = b * n, 0
            while a < n - 1:
                d = int(c.tokens[t + a + 1])
                if not float(c.accept_u[t + a + 1]) * float(q[t + a, d]) < float(p[t + a, d]):
                    break
                a += 1
            w = p[t + a].double()
            if a < n - 1:
                w = (w - q[t + a].double()).clamp(min=0)
            s = torch.cumsum(w, 0)
            assert (stay[b], keep[b]) == (a, t + a + 1)
            assert token[b] == int((s <= float(c.sample_u[b]) * s[-1]).sum())
        again, _ = c.run()
        assert again == [stay, token, keep]


def test_draws_at_the_ends():
    """Random numbers at and outside the ends, weights at the row's ends and around tile borders."""
    g = np.random.default_rng(23)
    for vocab in (1, 5, 1024, 1025, 4100):
        for spot in {0, vocab // 2, vocab - 1, min(1023, vocab - 1), min(1024, vocab - 1)}:
            c = Case(g, [1] * 6, vocab)
            c.p.zero_()
            c.p[:, spot] = 0.75
            c.sample_u.copy_(torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, float("nan")]))
            got, status = c.run()
            assert got[1] == [spot] * 6 and status == 0
            if spot > 0:
                c.p[:, 0] = 0.25
                got, _ = c.run()
                assert got[1] == [0, spot, spot, spot, 0, 0]
                c.sample_u.copy_(torch.tensor([0.25, 0.25 - 2.0 ** -25, 0.2, 0.5, 0.3, 0.0]))
                assert c.run()[0][1] == [spot, 0, 0, spot, spot, 0]


def test_borders_of_the_test_are_exact():
    """u q = p refuses, the next smaller u does not: products of 48 bits compared whole."""
    c = Case(np.random.default_rng(24), [2, 2, 2, 2], 3)
    c.tokens.fill_(1)
    p = np.float32(1 / 3) * np.float32(0.7)
    c.q.fill_(0.7)
    c.p.fill_(float(p))
    u = np.float32(1 / 3)
    exact = [float(np.float64(u) * np.float64(np.float32(0.7))) < float(p) for u in
             (u, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(0)), np.float32(0.34))]
    c.accept_u[1::2] = torch.tensor([u, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(0)),
                                     0.34])
    assert c.run()[0][0] == [int(x) for x in exact] and len(set(exact)) == 2
    c.q.fill_(0.5)
    c.p.fill_(0.25)
    c.accept_u.fill_(0.5)
    assert c.run()[0][0] == [0] * 4
    c.accept_u.fill_(0.5 - 2.0 ** -25)
    assert c.run()[0][0] == [1] * 4


def test_nothing_left_beside_the_drafter():
    """q at least p everywhere but for the draft, refused: the token comes from p."""
    g = np.random.default_rng(25)
    for vocab in (9, 3000):
        c = Case(g, [3, 2, 4], vocab)
        c.q.copy_((c.p * 1.5).clamp(max=1))
        c.accept_u.fill_(0.99)
        got, status = c.run()
        assert got == c.want() and status == 0 and got[0] == [0, 0, 0]
        # a certain token, looked up and refused, had all the weight
        c.q = None
        c.p.zero_()
        c.p[:, 4] = 0.5
        c.tokens.fill_(4)
        assert c.run()[0][1] == [4, 4, 4] == c.want()[1]


def test_bad_values_tokens_and_rows():
    g = np.random.default_rng(26)
    c = Case(g, [3, 2, 4, 2], 50)
    c.tokens[1], c.tokens[4] = -1, 50                            # first drafts of the first two
    got, status = c.run()
    assert got == c.want() and status == BAD_INDEX and got[0][:2] == [0, 0]
    c.q = None
    got, status = c.run()
    assert got == c.want() and status == BAD_INDEX
    # no weight anywhere; negative and NaN entries have none
    c = Case(g, [1, 1, 1], 50, drafter=False)
    c.p[0] = 0
    c.p[1] = -c.p[1]
    c.p[2, 7:] = float("nan")
    got, status = c.run()
    assert got[1][:2] == [-1, -1] and got == c.want() and status == BAD_VALUE
    c.p.fill_(float("nan"))
    assert c.run()[0][1] == [-1] * 3
    # rows that weigh more than a probability: some token of the vocabulary
    c = Case(g, [2] * 8, 5000)
    c.p.fill_(float("inf"))
    got, _ = c.run()
    assert all(0 <= t < 5000 for t in got[1])


def test_sequences_without_rows_or_pages():
    g = np.random.default_rng(27)
    c = Case(g, [3, 2, 4], 60)
    want = c.want()
    c.chunk.pos[3:5] = -1                                        # refused by the plan
    got, status = c.run()
    for x, y, none in zip(got, want, (0, -1, -1)):
        assert x == [y[0], none, y[2]]
    assert status == 0
    good = c.chunk.start.clone()
    for bad, flags in (([0, 3, 2, 9], [1]), ([0, 3, 5, 12], [2]), ([-2, 3, 5, 9], [0])):
        c.chunk.start.copy_(i32(bad))
        got, status = c.run()
        assert status == BAD_LENGTH
        for b in flags:
            assert [x[b] for x in got] == [0, -1, -1]
    c.chunk.start.copy_(good)
    empty = Case(g, [], 60)
    assert empty.run(se.workspace(se.se_draft_verify_workspace(1, 60))) == ([[], [], []], 0)


def test_one_workspace_for_calls_of_any_shape():
    g = np.random.default_rng(28)
    ws = se.workspace(max(se.se_draft_verify_workspace(b, v) for b, v in ((300, 40), (2, 70000), (8192, 1))))
    for rows, vocab in (([2] * 300, 40), ([2, 3], 70000), ([4] * 17, 900), ([1] * 8192, 1), ([3], 20000)):
        c = Case(g, rows, vocab)
        got, status = c.run(ws)
        assert got == c.want() and status == 0
        assert not ws[256:256 + 8192 * 4].any()


def test_replayed_from_a_graph_and_on_another_stream():
    g = np.random.default_rng(29)
    c = Case(g, [5, 1, 3], 4000)
    ws = se.workspace(se.se_draft_verify_workspace(3, 4000))
    c.run(ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        se.se_draft_verify(c.p, c.q, c.tokens, c.accept_u, c.sample_u, c.chunk, 3, *c.out, ws)
    for _ in range(4):
        c.accept_u.copy_(torch.from_numpy(g.random(9).astype(np.float32)))
        c.sample_u.copy_(torch.from_numpy(g.random(3).astype(np.float32)))
        graph.replay()
        assert [x.tolist() for x in c.out] == c.want()
    side = torch.cuda.Stream()
    for x in c.out:
        x.fill_(9)
    side.wait_stream(torch.cuda.current_stream())
    c.run(ws, stream=side)
    side.synchronize()
    assert [x.tolist() for x in c.out] == c.want()
