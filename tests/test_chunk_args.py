"""The chunk operators' argument checks (all on the host, before any CUDA call)."""
import ctypes

import pytest
import torch

from kv_cache_decode_quest_gb300 import binding, build

FAKE = 1 << 20                      # never dereferenced: validation fails first
P = ctypes.c_void_p(FAKE)
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def pool(**kw):
    c = binding.PagePoolC(FAKE, FAKE, FAKE, FAKE, FAKE, 10, 4)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def chunk(**kw):
    c = binding.ChunkC(FAKE, FAKE, FAKE, FAKE, 32)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def paged(**kw):
    c = binding.PagedKVC(FAKE, FAKE, None, FAKE, FAKE, 10, 4, 4, 128, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


BAD_POOLS = [dict(free_pages=None), dict(n_free=None), dict(n_pages=None), dict(block_table=None),
             dict(ctx_len=None), dict(num_pages=0), dict(max_pages_per_seq=0)]


def test_plan(lib):
    def call(p=pool(), new=P, batch=2, c=chunk(), ws=P, nbytes=512):
        return lib.se_chunk_plan(p, new, batch, c, ws, nbytes, None)
    for bad in BAD_POOLS:
        assert call(p=pool(**bad)) == INVALID, bad
    assert call(p=pool(num_pages=1 << 28)) == UNSUPPORTED
    assert call(p=pool(max_pages_per_seq=1 << 28)) == UNSUPPORTED
    assert call(p=None) == INVALID and call(c=None) == INVALID and call(new=None) == INVALID
    for bad in (dict(start=None), dict(seq=None), dict(pos=None), dict(slot=None),
                dict(max_tokens=-1)):
        assert call(c=chunk(**bad)) == INVALID, bad
    assert call(c=chunk(max_tokens=(1 << 24) + 1)) == UNSUPPORTED
    assert call(batch=-1) == INVALID
    assert call(ws=None) == WORKSPACE and call(nbytes=256) == WORKSPACE
    assert call(ws=ctypes.c_void_p(FAKE + 16)) == WORKSPACE
    assert lib.se_page_pool_workspace(1) == 512 and lib.se_page_pool_workspace(-1) == 0


def test_release(lib):
    def call(p=pool(), done=P, batch=2, ws=P, nbytes=512):
        return lib.se_pages_release(p, done, batch, ws, nbytes, None)
    for bad in BAD_POOLS:
        assert call(p=pool(**bad)) == INVALID, bad
    assert call(done=None) == INVALID and call(batch=-1) == INVALID
    assert call(ws=None) == WORKSPACE and call(nbytes=511) == WORKSPACE
    assert call(done=None, batch=0) == 0


def test_append(lib):
    def call(kv=paged(), k=P, v=P, stride=0, c=chunk(), batch=2, ws=P, nbytes=256):
        return lib.se_kv_append_chunk(kv, k, v, stride, c, batch, ws, nbytes, None)
    assert call(kv=paged(k=None)) == INVALID and call(kv=paged(block_table=None)) == INVALID
    assert call(kv=paged(head_dim=96)) == UNSUPPORTED and call(kv=paged(page_size=8)) == UNSUPPORTED
    assert call(k=None) == INVALID and call(v=None) == INVALID
    assert call(k=ctypes.c_void_p(FAKE + 8)) == INVALID
    assert call(v=ctypes.c_void_p(FAKE + 8)) == INVALID
    assert call(stride=511) == INVALID and call(stride=516) == INVALID and call(stride=-512) == INVALID
    assert call(batch=-1) == INVALID and call(c=chunk(seq=None)) == INVALID
    assert call(ws=None) == WORKSPACE and call(nbytes=255) == WORKSPACE
    assert call(k=None, v=None, batch=0) == 0
    assert call(k=None, v=None, c=chunk(max_tokens=0, seq=None, pos=None, slot=None)) == 0


def test_attn(lib):
    need = lib.se_chunk_attn_workspace(2, 32, 4, 32, 128)
    assert need >= 256 and need % 256 == 0

    def opts(**kw):
        o = binding.ChunkAttnOptsC(0, 0, 0, 0, None, None)
        for k, v in kw.items():
            setattr(o, k, v)
        return ctypes.byref(o)

    def call(kv=paged(), q=P, c=chunk(), batch=2, hq=32, scale=0.1, o=None, out=P, ws=P,
             nbytes=need):
        return lib.se_chunk_attn(kv, q, c, batch, hq, scale, o, out, None, ws, nbytes, None)
    assert call(kv=paged(v=None)) == INVALID and call(kv=paged(ctx_len=None)) == INVALID
    assert call(kv=paged(head_dim=80)) == UNSUPPORTED and call(kv=paged(page_size=32)) == UNSUPPORTED
    assert call(kv=paged(max_pages_per_seq=1 << 28)) == UNSUPPORTED
    assert call(hq=12) == UNSUPPORTED and call(hq=30) == UNSUPPORTED and call(hq=0) == INVALID
    assert call(q=None) == INVALID and call(out=None) == INVALID and call(c=None) == INVALID
    assert call(q=ctypes.c_void_p(FAKE + 2)) == INVALID
    assert call(out=ctypes.c_void_p(FAKE + 8)) == INVALID
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert call(scale=bad) == INVALID
    for bad in (dict(out_dtype=2), dict(window=-1), dict(sink=-1), dict(q_stride=4088),
                dict(q_stride=4100), dict(q_stride=-4096)):
        assert call(o=opts(**bad)) == INVALID, bad
    assert call(c=chunk(max_tokens=(1 << 24) + 1)) == UNSUPPORTED
    assert call(batch=-1) == INVALID
    assert call(batch=8193) == UNSUPPORTED
    assert call(kv=paged(max_pages_per_seq=(1 << 26) + 1)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(nbytes=need - 1) == WORKSPACE
    assert call(q=None, out=None, batch=0) == 0
    assert call(q=None, out=None, c=chunk(max_tokens=0, seq=None, pos=None, slot=None)) == 0
    for bad in ((-1, 32, 4, 32, 128), (1, -1, 4, 32, 128), (1, 32, 0, 32, 128), (1, 32, 4, 30, 128),
                (1, 32, 4, 32, 96), (1, 32, 4, 12, 128), (1, (1 << 24) + 1, 4, 32, 128)):
        assert lib.se_chunk_attn_workspace(*bad) == 0, bad


def test_binding_refuses_layouts_it_cannot_pass(lib):
    x = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    assert binding._token_stride(x, "x") == 512
    assert binding._token_stride(torch.zeros(4, 12, 128)[:, 4:8], "x") == 1536
    for bad in (x.transpose(1, 2), x[:, :, ::2], x[:, ::2], x.view(16, 128)):
        with pytest.raises(binding.SparseEngineError):
            binding._token_stride(bad, "x")


def test_binding_refuses_rows_that_are_not_there(lib):
    """Expanded or too short tensors never reach the library (every pointer here is a CPU one)."""
    with pytest.raises(binding.SparseEngineError, match="overlap"):
        binding._token_stride(torch.zeros(1, 4, 128).expand(8, 4, 128), "x")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    kv = binding.PagedKV(z(4, 2, 16, 64), z(4, 2, 16, 64), None, i(2, 4), i(2))
    c = binding.Chunk.empty(2, 8, "cpu")
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    good = z(8, 2, 64)
    for bad in (z(7, 2, 64), z(8, 4, 64), z(8, 1, 64), z(8, 2, 128)):
        for k, v in ((bad, bad), (good, z(7, 2, 64))):
            with pytest.raises(binding.SparseEngineError, match="needed|differ"):
                binding.se_kv_append_chunk(kv, k, v, c, 2, ws, stream=NoStream)
    for bad in (z(7, 4, 64), z(8, 2, 64), z(8, 4, 128), z(1, 4, 64).expand(8, 4, 64)):
        with pytest.raises(binding.SparseEngineError, match="needed|overlap"):
            binding.se_chunk_attn(kv, bad, c, 2, 4, 1.0, z(8, 4, 64), None, ws, stream=NoStream)

    q = z(8, 4, 64)
    for out, f32 in ((z(7, 4, 64), 0), (z(8, 4, 64), 1), (z(8, 4, 128)[:, :, :64], 0),
                     (torch.zeros(8, 4, 64), 0)):
        with pytest.raises(binding.SparseEngineError, match="needed|contiguous"):
            binding.se_chunk_attn(kv, q, c, 2, 4, 1.0, out, None, ws, out_dtype=f32,
                                  stream=NoStream)
    for lse in (torch.zeros(7, 4), torch.zeros(8, 8)[:, :4]):
        with pytest.raises(binding.SparseEngineError, match="lse"):
            binding.se_chunk_attn(kv, q, c, 2, 4, 1.0, q.clone(), lse, ws, stream=NoStream)



class NoStream:
    cuda_stream = None


def test_attn_wait_limit(lib):
    need = lib.se_chunk_attn_workspace(2, 32, 4, 32, 128)
    for limit, rc in ((-1, INVALID), (-2 ** 31, INVALID), (0, 0), (1, 0), (2 ** 31 - 1, 0)):
        o = binding.ChunkAttnOptsC(0, 0, 0, 0, None, None, limit)
        empty = chunk(max_tokens=0, seq=None, pos=None, slot=None)
        assert lib.se_chunk_attn(paged(), None, empty, 2, 32, 0.1, ctypes.byref(o), None, None, P,
                                 need, None) == rc, limit


def chunk_of(rows=8, batch=2, **kw):
    t = dict(start=torch.zeros(batch + 1, dtype=torch.int32),
             **{x: torch.zeros(rows, dtype=torch.int32) for x in ("seq", "pos", "slot")})
    return binding.Chunk(**{**t, **kw})


def pool_of(batch=2, **kw):
    p = binding.PagePool.empty(batch, 6, 4, "cpu")
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def cache_of(batch=2, dtype=torch.bfloat16, meta=None):
    z = torch.zeros(4, 2, 16, 64, dtype=dtype)
    return binding.PagedKV(z, z.clone(), meta, torch.zeros(batch, 4, dtype=torch.int32),
                           torch.zeros(batch, dtype=torch.int32))


def test_binding_refuses_integers_of_another_type(lib):
    """A bool, int64 or strided table of a holder is refused, also when it is put there later."""
    good, ws = torch.zeros(8, dtype=torch.int32), torch.zeros(1 << 10, dtype=torch.uint8)

    def plan(p, c):
        binding.se_chunk_plan(p, good, 2, c, ws, stream=NoStream)
    for bad in (good.bool(), good.long(), good.short(), good.float(),
                torch.zeros(16, dtype=torch.int32)[::2]):
        for field in ("start", "seq", "pos", "slot"):
            with pytest.raises(binding.SparseEngineError, match=f"Chunk.{field}.*int32"):
                plan(pool_of(), chunk_of(**{field: bad}))
        for field in ("free_pages", "n_free", "n_pages", "ctx_len"):
            with pytest.raises(binding.SparseEngineError, match=f"PagePool.{field}.*int32"):
                plan(pool_of(**{field: bad}), chunk_of())
        with pytest.raises(binding.SparseEngineError, match="PagePool.block_table.*int32"):
            plan(pool_of(block_table=bad.view(2, 4) if bad.is_contiguous() else bad[:, None]),
                 chunk_of())
    c = chunk_of()
    with pytest.raises(binding.SparseEngineError, match="workspace"):       # all that is wrong here
        binding.se_chunk_plan(pool_of(), good, 2, c, ws[:8], stream=NoStream)
    c.pos = c.pos.long()
    with pytest.raises(binding.SparseEngineError, match="Chunk.pos.*int32"):
        plan(pool_of(), c)


def test_binding_refuses_tables_that_are_too_short(lib):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    refused = lambda m: pytest.raises(binding.SparseEngineError, match=m)

    def plan(pool=None, new=i(2), batch=2, c=None):
        binding.se_chunk_plan(pool or pool_of(), new, batch, c or chunk_of(), ws, stream=NoStream)

    def release(pool=None, done=i(2), batch=2):
        binding.se_pages_release(pool or pool_of(), done, batch, ws, stream=NoStream)
    for bad in (i(1), torch.zeros(2, dtype=torch.bool), torch.zeros(2, dtype=torch.int64), i(4)[::2]):
        with refused("new_len.*int32"):
            plan(new=bad)
        with refused("done.*int32"):
            release(done=bad)
    for bad in (dict(n_pages=i(1)), dict(ctx_len=i(1)), dict(block_table=i(1, 4)), dict(n_free=i(0))):
        with refused("PagePool.*too short for 2 sequences|n_free: one word"):
            plan(pool_of(**bad))
        with refused("PagePool.*too short for 2 sequences|n_free: one word"):
            release(pool_of(**bad))
    kv, q, k = cache_of(), torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64).bfloat16()
    for bad in (chunk_of(pos=i(7)), chunk_of(slot=i(7)), chunk_of(start=i(2))):
        with refused("Chunk.*too short for 2 sequences|Chunk: fewer entries"):
            plan(c=bad)
        with refused("Chunk.*too short for 2 sequences|Chunk: fewer entries"):
            binding.se_chunk_attn(kv, q, bad, 2, 4, 1.0, q.clone(), None, ws, stream=NoStream)
    for bad in (chunk_of(pos=i(7)), chunk_of(slot=i(7))):
        with refused("Chunk.*too short for 2 sequences|Chunk: fewer entries"):
            binding.se_kv_append_chunk(kv, k, k, bad, 2, ws, stream=NoStream)
    three = chunk_of(batch=3)
    with refused("PagedKV.*too short for 3 sequences"):
        binding.se_kv_append_chunk(kv, k, k, three, 3, ws, stream=NoStream)
    with refused("PagedKV.*too short for 3 sequences"):
        binding.se_chunk_attn(kv, q, three, 3, 4, 1.0, q.clone(), None, ws, stream=NoStream)


def test_binding_refuses_numbers_of_another_type(lib):
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    kv, c = cache_of(), chunk_of()
    q, k = torch.zeros(8, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 64, dtype=torch.bfloat16)

    def attn(kv=kv, q=q, out=q.clone(), lse=None, f32=0):
        binding.se_chunk_attn(kv, q, c, 2, 4, 1.0, out, lse, ws, out_dtype=f32, stream=NoStream)

    def append(kv=kv, k=k, v=k):
        binding.se_kv_append_chunk(kv, k, v, c, 2, ws, stream=NoStream)
    for dt in (torch.float16, torch.float32, torch.int16):
        for call in (lambda: attn(q=q.to(dt)), lambda: append(k=k.to(dt)), lambda: append(v=k.to(dt)),
                     lambda: attn(kv=cache_of(dtype=dt)), lambda: append(kv=cache_of(dtype=dt)),
                     lambda: append(kv=cache_of(meta=torch.zeros(2, 4, 2, 2, 64, dtype=dt)))):
            with pytest.raises(binding.SparseEngineError, match="bfloat16"):
                call()
    for out, f32 in ((q.half(), 0), (q.short(), 0), (q.int(), 1), (q.float(), 0), (q, 1)):
        with pytest.raises(binding.SparseEngineError, match="out_dtype"):
            attn(out=out, f32=f32)
    for lse in (torch.zeros(8, 4, dtype=torch.float64), torch.zeros(8, 4, dtype=torch.int32)):
        with pytest.raises(binding.SparseEngineError, match="float32 lse"):
            attn(lse=lse)
