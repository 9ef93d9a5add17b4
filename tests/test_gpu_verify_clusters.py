"""GPU parity of the draft verification where two to eight blocks, or more, share a sequence: every integer
equal to the definition's in 64 bits (a draw on a border has a chance below 10^-6)."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from tests.test_gpu_verify import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def case(rows, vocab, dtype, drafter, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(rows)
    c = Case.__new__(Case)
    c.rows, c.vocab = rows, vocab

    def soft():
        x = torch.full((n, vocab + pad), float("nan"), device="cuda")
        x[:, :vocab] = torch.softmax(3 * torch.randn(n, vocab, generator=g, device="cuda"), 1)
        return x.to(dtype)[:, :vocab]
    c.p, c.q = soft(), soft() if drafter else None
    c.tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    c.accept_u, c.sample_u = (torch.rand(k, generator=g, device="cuda") for k in (n, len(rows)))
    c.accept_u[torch.rand(n, generator=g, device="cuda") < 0.6] = 0
    c.chunk = se.Chunk.empty(len(rows), n)
    c.chunk.start.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(rows)])))
    c.chunk.pos.copy_(7 * torch.arange(n, device="cuda"))
    c.out = [torch.full((len(rows),), 55, dtype=torch.int32, device="cuda") for _ in range(3)]
    return c


def want(c):
    got, at = [], 0
    for b, n in enumerate(c.rows):
        if n == 0:
            got.append((0, -1, -1))
            continue
        a, p = 0, c.p[at:at + n].double()
        q = None if c.q is None else c.q[at:at + n].double()
        while a < n - 1:
            d = int(c.tokens[at + a + 1])
            if not float(c.accept_u[at + a + 1]) * (1.0 if q is None else float(q[a, d])) < float(p[a, d]):
                break
            a += 1
        w = p[a].clone()
        if a < n - 1 and q is not None:
            w = (w - q[a]).clamp(min=0)
        elif a < n - 1:
            w[int(c.tokens[at + a + 1])] = 0
        if float(w.sum()) == 0:
            w = p[a]
        s = torch.cumsum(w, 0)
        got.append((a, int((s <= float(c.sample_u[b]) * s[-1]).sum()), 7 * at + 1 + a))
        at += n
    return [list(x) for x in zip(*got)]


# vocabulary and sequences: blocks of a sequence 2, 3, 7, 8, 8 and, where a grid has no more, 6 or 2; more
# than 8 (a counter)
SHAPES = [(9000, [3, 2, 4]), (20001, [2, 0, 3, 0, 0, 5]), (50002, [4, 1, 2, 3]), (65000, [0, 3, 3]),
          (63997, [2] * 17), (50000, [2, 3, 0] * 33 + [1]), (20000, [2, 1, 0, 3] * 63), (131072, [3, 0, 2]),
          (90001, [2, 4])]


@pytest.mark.parametrize("vocab,rows", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
def test_every_split(vocab, rows, dtype, drafter):
    ws = se.workspace(se.se_draft_verify_workspace(len(rows), vocab))
    for pad in (0, 3):
        c = case(rows, vocab, dtype, drafter, vocab + pad, pad)
        expect = want(c)
        for _ in range(2):
            got, status = c.run(ws)
            assert got == expect and status == 0
    assert not ws[256:256 + 8192 * 4].any()


@pytest.mark.parametrize("vocab,rows", [(9000, [3, 2, 4]), (20001, [2, 0, 3, 0, 0, 5]), (65000, [3, 3, 2]),
                                        (50000, [2, 3, 0] * 33 + [1]), (131072, [3, 0, 2])])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nothing_left_and_no_weight(vocab, rows, dtype):
    """Every first draft refused with q above p everywhere: the token comes from p; rows of zeros have none;
    the same workspace serves the calls behind."""
    ws = se.workspace(se.se_draft_verify_workspace(len(rows), vocab))
    c = case(rows, vocab, dtype, True, vocab + 1)
    expect, p, q = want(c), c.p, c.q
    c.q = (p * 2).clamp(max=1)
    c.accept_u.fill_(0.99)
    for _ in range(2):
        got, status = c.run(ws)
        assert got == want(c) and status == 0 and got[0] == [0] * len(rows)
    c.p = torch.zeros_like(p)
    got, status = c.run(ws)
    assert status == 16 and got[1] == [-1] * len(rows) and not any(got[0])
    ws[:4] = 0
    # some without weight beside some with it
    c.p = p.clone()
    first = int(np.flatnonzero(rows)[0])
    c.p[:rows[first]] = 0
    got, status = c.run(ws)
    rest = want(c)
    assert status == 16 and got[1][first] == -1
    for b in range(len(rows)):
        assert b == first or [x[b] for x in got] == [x[b] for x in rest]
    ws[:4] = 0
    c = case(rows, vocab, dtype, True, vocab + 1)
    got, status = c.run(ws)
    assert got == expect and status == 0 and not ws[256:256 + 8192 * 4].any()
