"""A wait inside se_chunk_attn that runs out: status, return, and the calls after it."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from tests.test_gpu_chunk import Attn, held

pytestmark = pytest.mark.gpu
TIMEOUT = 8


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def test_wait_that_runs_out_reports_timeout_and_returns():
    """A limit of 1 ns gives up at a wait's first failed try (about 4 us).  The wait that fails is one
    for the next piece of work: eight sequences have rows, with 500 empty ones between them, and a
    block whose share goes from one to the next has its softmax and MMA warps wait while
    those are passed over (16 dependent reads of lengths, over 10 us).  Its producer
    still finds the piece and begins its copies, which have to land before the block leaves."""
    g = np.random.default_rng([51])
    B, H, G, D = 4000, 4, 2, 64
    ctx, new = [0] * B, [0] * B
    for i in range(8):
        ctx[500 * i + 250], new[500 * i + 250] = 5600 + 131 * i, 1
    c = held(g, B, H, D, ctx, new)
    chunk = c.add(new)
    a = Attn(c, G)
    a.run(chunk)
    a.check(chunk)
    out, lse = a.out.clone(), a.lse.clone()
    se.se_chunk_attn(c.kv, a.qt, chunk, B, a.Hq, a.scale, a.out, a.lse, a.ws, wait_limit_ns=1)
    torch.cuda.synchronize()
    assert se.status_word(a.ws) & TIMEOUT
    a.ws.zero_()
    a.out.fill_(7)
    a.lse.fill_(7)
    a.call(chunk)
    a.check(chunk)
    assert torch.equal(a.out, out) and torch.equal(a.lse, lse)
    # a limit that nothing reaches changes nothing
    a.out.fill_(7)
    se.se_chunk_attn(c.kv, a.qt, chunk, B, a.Hq, a.scale, a.out, a.lse, a.ws,
                     wait_limit_ns=2 ** 31 - 1)
    assert se.status_word(a.ws) == 0 and torch.equal(a.out, out) and torch.equal(a.lse, lse)
