"""The rotation, append, carry and verification calls where offsets pass 32 bits: caches, summaries and
rows of more than 2^32 elements, work at their ends."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from tests.test_gpu_chunk import i32
from tests.test_gpu_rope import bf16, make, marked, small_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    yield lib
    torch.cuda.empty_cache()


def test_append_and_carry_at_the_end_of_a_large_cache():
    g = np.random.default_rng(51)
    P, H, D, B, maxp, L = 270000, 8, 128, 64, 33000, 500
    shape = (P, H, 16, D)
    assert np.prod(shape, dtype=np.int64) > 1 << 32 and B * maxp * H * 2 * D > 1 << 32
    kv = se.PagedKV(*(torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)),
                    torch.empty(B, maxp, H, 2, D, dtype=torch.bfloat16, device="cuda"),
                    torch.full((B, maxp), -1, dtype=torch.int32, device="cuda"), i32([0] * B))
    small = se.PagedKV(*(torch.zeros(100, H, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)),
                       torch.zeros(1, 40, H, 2, D, dtype=torch.bfloat16, device="cuda"),
                       i32(range(100))[:40].view(1, 40).contiguous(), i32([0]))
    n = -(-L // 16)
    b, far = B - 1, maxp - n - 2                          # the last sequence, its last pages
    pages = P - 1 - torch.arange(n, dtype=torch.int32, device="cuda")
    kv.block_table[b, far:far + n] = pages
    t = torch.arange(L, device="cuda")
    rope = make(g, 128, 128, 0, (1, 1))
    x = bf16(g, L, 4 + 2 * H, D)
    q, k, v = x[:, :4], x[:, 4:4 + H], x[:, 4 + H:]
    pos = (far * 16 + t).int()
    chunk = se.Chunk(i32([0] * B + [L]), torch.full_like(pos, b), pos, (pages[t // 16] * 16 + t % 16).int())
    qo, ko = marked(L, 4, D), marked(L, H, D)
    ws = small_ws()
    se.se_rope_append_chunk(kv, rope, q, k, v, qo, chunk, B, ws)
    se.se_qk_rope(rope, pos, q, k, q.clone(), ko, ws)
    one = se.Chunk(i32([0, L]), torch.zeros_like(pos), t.int(), t.int())
    se.se_kv_append_chunk(small, ko, v.contiguous(), one, 1, ws)
    assert se.status_word(ws) == 0 and int(kv.ctx_len[b]) == far * 16 + L
    last = L % 16
    for a, c in ((kv.k, small.k), (kv.v, small.v)):
        assert a[pages[:n - 1].long()].equal(c[:n - 1])
        assert a[pages[n - 1].long(), :, :last].equal(c[n - 1, :, :last])
    assert kv.meta[b, far:far + n].equal(small.meta[0, :n])
    # the last page's rows into a page of its own, its summary folded anew
    to, old = P - 3 * n, int(pages[n - 1])
    kv.block_table[b, far + n - 1] = to
    kv.meta[b, far + n - 1] = 0
    c = se.Carry(i32([-1] * B), i32([-1] * b + [old]))
    se.se_pages_carry(kv, c, B, ws)
    assert se.status_word(ws) == 0
    assert kv.k[to, :, :last].equal(small.k[n - 1, :, :last])
    assert kv.meta[b, far + n - 1].equal(small.meta[0, n - 1])
    # another sequence takes all its summaries over
    kv.ctx_len[b - 1] = far * 16 + L
    kv.block_table[b - 1] = kv.block_table[b]
    se.se_pages_carry(kv, se.Carry(i32([-1] * (b - 1) + [b, -1]), i32([-1] * B)), B, ws)
    assert kv.meta[b - 1, far:far + n - 1].equal(small.meta[0, :n - 1])
    assert se.status_word(ws) == 0


def test_rows_past_32_bits():
    g = np.random.default_rng(52)
    rows, heads, D = 900000, 40, 128
    assert rows * heads * D > 1 << 32
    rope = make(g, 64, D, 1, (1, 0))
    x = torch.empty(rows, heads, D, dtype=torch.bfloat16, device="cuda")
    tail = bf16(g, 100, heads, D)
    x[-100:] = tail
    pos = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    pos[-100:] = torch.arange(100, device="cuda")
    se.se_qk_rope(rope, pos, x, None, x, None, small_ws())
    want = marked(100, heads, D)
    se.se_qk_rope(rope, pos[-100:].contiguous(), tail, None, want, None, small_ws())
    assert x[-100:].equal(want)


def test_probabilities_past_32_bits():
    g = torch.Generator(device="cuda").manual_seed(53)
    rows, V = 33000, 131072
    assert rows * V > 1 << 32
    p, q = (torch.empty(rows, V, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 5
    for t in (p, q):
        t[-n:] = torch.softmax(3 * torch.randn(n, V, generator=g, device="cuda"), 1).bfloat16()
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    au, su = torch.zeros(rows, device="cuda"), torch.tensor([0.3], device="cuda")
    out = [i32([9]) for _ in range(3)]
    chunk = se.Chunk(i32([rows - n, rows]), torch.zeros_like(tok), torch.arange(rows, device="cuda").int(),
                     torch.zeros_like(tok))
    ws = se.workspace(se.se_draft_verify_workspace(1, V))
    se.se_draft_verify(p, q, tok, au, su, chunk, 1, *out, ws)
    few = se.Chunk(i32([0, n]), torch.zeros(n, dtype=torch.int32, device="cuda"),
                   chunk.pos[-n:].contiguous(), torch.zeros(n, dtype=torch.int32, device="cuda"))
    got = [x.tolist() for x in out]
    se.se_draft_verify(p[-n:].clone(), q[-n:].clone(), tok[-n:].contiguous(), au[-n:].contiguous(), su, few,
                       1, *out, ws)
    assert got == [x.tolist() for x in out] and se.status_word(ws) == 0
