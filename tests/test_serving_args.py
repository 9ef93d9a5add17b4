"""Argument checks of the rotation, verification, fork and truncation calls (all on the host, before any
CUDA call)."""
import ctypes
import math

import pytest
import torch

from kv_cache_decode_quest_gb300 import binding, build
from oracle import rope as orope
from tests.test_chunk_args import (BAD_POOLS, FAKE, INVALID, NoStream, P, UNSUPPORTED, WORKSPACE,
                                   cache_of, chunk, chunk_of, paged, pool, pool_of)

ODD = ctypes.c_void_p(FAKE + 8)
Error = binding.SparseEngineError


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def rope(**kw):
    c = binding.RopeC(FAKE, 64, 0, 1.0, 1e-6, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def carry(**kw):
    c = binding.PageCarryC(FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


BAD_ROPES = [dict(turns=None), dict(turns=FAKE + 4), dict(rot_dim=-16), dict(rot_dim=144),
             dict(rot_dim=8), dict(rot_dim=72), dict(layout=2), dict(layout=-1),
             dict(amplitude=math.nan), dict(amplitude=math.inf), dict(eps=-1e-6), dict(eps=math.nan),
             dict(q_weight=FAKE + 2), dict(k_weight=FAKE + 8)]


# ---------------------------------------------------------------------------
# the C entry points
# ---------------------------------------------------------------------------

def test_turns_of_every_scaling(lib):
    for kind in range(5):
        for rot, base in ((16, 1e4), (128, 1e4), (96, 5e5), (64, 1.5)):
            args = (8.0, 4096.0, 1.0, 32.0 if kind == binding.SE_ROPE_YARN else 4.0)
            turns, amp = binding.se_rope_turns(rot, base, kind, *args)
            want, want_amp = orope.frequencies(base, rot, kind, *args)
            assert turns.shape == (rot // 2,) and abs(amp - want_amp) <= 2.0 ** -24 * want_amp
            for t, f in zip(turns.tolist(), want):
                # a few roundings to 53 bits on either side
                assert abs((t % 2 ** 64) * 2 * math.pi / 2 ** 64 - f) <= 16 * 2.0 ** -53 * f + 2.0 ** -60


def test_turns_refused(lib):
    def call(base=1e4, rot=64, s=None, out=(ctypes.c_uint64 * 64)()):
        return lib.se_rope_turns(base, rot, None if s is None else ctypes.byref(s), out, None)
    assert call() == 0 and call(rot=128) == 0
    for bad in (dict(base=1.0), dict(base=0.5), dict(base=math.nan), dict(base=math.inf), dict(rot=0),
                dict(rot=8), dict(rot=144), dict(rot=40), dict(out=None)):
        assert call(**bad) == INVALID, bad
    S = binding.RopeScalingC
    for bad in (S(5, 2, 4096, 1, 32), S(-1, 2, 4096, 1, 32), S(1, 0.5, 0, 0, 0), S(1, math.nan, 0, 0, 0),
                S(2, math.inf, 0, 0, 0), S(3, 2, 0, 1, 32), S(3, 2, 4096, 0, 32), S(3, 2, 4096, 4, 4),
                S(4, 2, -1, 1, 4), S(4, 2, math.nan, 1, 4), S(4, 2, 4096, 4, 1)):
        assert call(s=bad) == INVALID, (bad.kind, bad.factor)
    assert call(s=S(0, math.nan, 0, 0, 0)) == 0                    # not looked at
    # a base that overflows
    assert call(base=1e300, s=S(2, 3e38, 0, 0, 0)) == INVALID


def test_qk_rope(lib):
    def call(r=rope(), pos=P, rows=4, hq=4, hk=2, dim=128, q=P, sq=0, k=P, sk=0, qo=P, so=0, ko=P,
             sko=0, ws=P, n=256):
        return lib.se_qk_rope(r, pos, rows, hq, hk, dim, q, sq, k, sk, qo, so, ko, sko, ws, n, None)
    for bad in BAD_ROPES:
        assert call(r=rope(**bad)) == INVALID, bad
    assert call(r=rope(), dim=96) == UNSUPPORTED and call(r=rope(rot_dim=128), dim=64) == INVALID
    assert call(r=None) == INVALID and call(pos=None) == INVALID and call(rows=-1) == INVALID
    assert call(rows=(1 << 24) + 1) == UNSUPPORTED and call(hq=1025) == UNSUPPORTED
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(q=ODD), dict(ko=ODD),
                dict(hq=-1), dict(hk=-1), dict(sq=511), dict(sq=516), dict(so=504), dict(sk=255),
                dict(sko=-256), dict(so=1024), dict(sk=1024)):       # (in place with two strides)
        assert call(**bad) == INVALID, bad
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE and call(ws=ODD) == WORKSPACE
    assert call(rows=0, pos=None, q=None, k=None) == 0


def test_rope_append(lib):
    def call(kv=paged(), r=rope(), q=P, sq=0, hq=8, k=P, v=P, s=0, qo=P, so=0, c=chunk(), batch=2, ws=P,
             n=256):
        return lib.se_rope_append_chunk(kv, r, q, sq, hq, k, v, s, qo, so, c, batch, ws, n, None)
    for bad in BAD_ROPES:
        assert call(r=rope(**bad)) == INVALID, bad
    assert call(kv=paged(k=None)) == INVALID and call(kv=paged(head_dim=96)) == UNSUPPORTED
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD),
                dict(q=ODD), dict(hq=-1), dict(s=511), dict(s=516), dict(sq=8), dict(so=2048),
                dict(batch=-1), dict(c=None), dict(c=chunk(slot=None))):
        assert call(**bad) == INVALID, bad
    assert call(hq=1025) == UNSUPPORTED and call(c=chunk(max_tokens=(1 << 24) + 1)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE
    assert call(batch=0, k=None, v=None, q=None, qo=None) == 0
    none = chunk(max_tokens=0, seq=None, pos=None, slot=None)
    assert call(c=none, k=None, v=None, q=None, qo=None) == 0


def test_verify(lib):
    need = lib.se_draft_verify_workspace(2, 1000)
    assert need >= 256 and need % 256 == 0

    def call(p=P, q=P, s=0, t=1, V=1000, tok=P, au=P, su=P, c=chunk(), batch=2, na=P, nt=P, kp=P, ws=P,
             n=need):
        return lib.se_draft_verify(p, q, s, t, V, tok, au, su, c, batch, na, nt, kp, ws, n, None)
    for bad in (dict(p=None), dict(p=ODD), dict(q=ODD), dict(s=999), dict(s=-1000), dict(t=2), dict(t=-1),
                dict(V=0), dict(tok=None), dict(au=None), dict(su=None), dict(c=None),
                dict(c=chunk(start=None)), dict(c=chunk(pos=None)), dict(c=chunk(max_tokens=-1)),
                dict(batch=-1), dict(na=None), dict(nt=None), dict(kp=None)):
        assert call(**bad) == INVALID, bad
    assert call(V=(1 << 22) + 1) == UNSUPPORTED and call(batch=8193) == UNSUPPORTED
    assert call(c=chunk(max_tokens=(1 << 24) + 1)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE and call(ws=ODD) == WORKSPACE
    assert call(batch=0, su=None) == 0
    for bad in ((-1, 10), (8193, 10), (1, 0), (1, (1 << 22) + 1)):
        assert lib.se_draft_verify_workspace(*bad) == 0, bad


def test_fork_and_truncate(lib):
    need = lib.se_pages_truncate_workspace(2, 10)
    assert need % 256 == 0 and need >= lib.se_page_pool_workspace(2) + 40

    def fork(p=pool(), refs=P, src=P, batch=2, c=carry(), ws=P, n=512):
        return lib.se_pages_fork(p, refs, src, batch, c, ws, n, None)

    def cut(p=pool(), refs=P, src=P, batch=2, c=carry(), ws=P, n=need):
        return lib.se_pages_truncate(p, refs, src, batch, c, ws, n, None)
    for call in (fork, cut):
        for bad in BAD_POOLS:
            assert call(p=pool(**bad)) == INVALID, bad
        for bad in (dict(src=None), dict(batch=-1), dict(c=None), dict(c=carry(from_seq=None)),
                    dict(c=carry(from_page=None)), dict(p=None)):
            assert call(**bad) == INVALID, bad
        assert call(batch=8193) == UNSUPPORTED and call(p=pool(num_pages=1 << 28)) == UNSUPPORTED
        # 2^30 entries of the block table are served, more are not
        assert call(p=pool(max_pages_per_seq=1 << 26), batch=16, ws=None) == WORKSPACE
        assert call(p=pool(max_pages_per_seq=1 << 26), batch=17) == UNSUPPORTED
        assert call(p=pool(max_pages_per_seq=(1 << 27) - 1), batch=9) == UNSUPPORTED
        assert call(ws=None) == WORKSPACE and call(n=511) == WORKSPACE and call(ws=ODD) == WORKSPACE
        assert call(batch=0, src=None) == 0
    assert fork(refs=None) == INVALID and cut(n=need - 1) == WORKSPACE
    for bad in ((-1, 10), (8193, 10), (1, 0), (1, 1 << 28)):
        assert lib.se_pages_truncate_workspace(*bad) == 0, bad


def test_carry(lib):
    def call(kv=paged(), c=carry(), batch=2, ws=P, n=256):
        return lib.se_pages_carry(kv, c, batch, ws, n, None)
    for bad in (dict(kv=paged(v=None)), dict(c=None), dict(c=carry(from_seq=None)), dict(batch=-1)):
        assert call(**bad) == INVALID, bad
    assert call(kv=paged(head_dim=80)) == UNSUPPORTED and call(batch=8193) == UNSUPPORTED
    assert call(kv=paged(max_pages_per_seq=(1 << 26) + 1)) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE and call(n=255) == WORKSPACE and call(batch=0) == 0


# ---------------------------------------------------------------------------
# the binding (every tensor here is a CPU one, so no call may reach a kernel)
# ---------------------------------------------------------------------------

def z(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


WS = torch.zeros(1 << 16, dtype=torch.uint8)


def refused(match):
    return pytest.raises(Error, match=match)


def test_binding_rope_holder(lib):
    def call(r):
        binding.se_qk_rope(r, i32(4), z(4, 2, 64), z(4, 1, 64), z(4, 2, 64), z(4, 1, 64), WS,
                           stream=NoStream)
    good = binding.Rope.make(64, device="cpu", q_weight=z(64), k_weight=z(64))
    with refused("current CUDA device"):
        call(good)
    with refused("turns.*int64"):
        call(binding.Rope(torch.zeros(32), 64))
    with refused("32 entries"):
        call(binding.Rope(torch.zeros(31, dtype=torch.int64), 64))
    with refused("32 entries"):
        call(binding.Rope(None, 64))
    for w in (z(64, dtype=torch.float32), z(1, 64), z(128)[::2]):
        with refused("q_weight.*bfloat16"):
            call(binding.Rope(None, 0, q_weight=w))
        with refused("k_weight.*bfloat16"):
            call(binding.Rope(None, 0, k_weight=w))
    for n in (32, 128):
        with refused(f"weights of {n} channels, heads of 64"):
            call(binding.Rope(None, 0, q_weight=z(n)))
    good.k_weight = z(16)
    with refused("two lengths"):
        call(good)
    with refused("invalid argument"):
        binding.Rope.make(40, device="cpu")


def test_binding_rope_rows(lib):
    r = binding.Rope.make(64, device="cpu")
    c, kv = chunk_of(), cache_of()

    def rows(pos=i32(8), q=z(8, 4, 64), k=z(8, 2, 64), qo=z(8, 4, 64), ko=z(8, 2, 64)):
        binding.se_qk_rope(r, pos, q, k, qo, ko, WS, stream=NoStream)

    def append(q=z(8, 4, 64), k=z(8, 2, 64), v=z(8, 2, 64), qo=z(8, 4, 64), kv=kv, c=c, batch=2):
        binding.se_rope_append_chunk(kv, r, q, k, v, qo, c, batch, WS, stream=NoStream)
    for call in (rows, append):
        with refused("current CUDA device"):
            call()
        with refused("current CUDA device"):
            call(q=None, qo=None)
        for bad in (dict(q=None), dict(qo=None)):
            with refused("without a tensor"):
                call(**bad)
        for bad in (dict(q=z(8, 4, 64, dtype=torch.float16)), dict(qo=z(8, 4, 64, dtype=torch.float32))):
            with refused("bfloat16"):
                call(**bad)
        for bad in (dict(q=z(7, 4, 64)), dict(qo=z(7, 4, 64)), dict(qo=z(8, 2, 64)),
                    dict(q=z(8, 64)), dict(q=z(8, 4, 128)[:, :, ::2]), dict(q=z(1, 4, 64).expand(8, 4, 64)),
                    dict(qo=z(1, 4, 64).expand(8, 4, 64)), dict(qo=z(4, 8, 64).transpose(0, 1))):
            with refused("needed|overlap"):
                call(**bad)
    for bad in (i32(16)[::2], torch.zeros(8, dtype=torch.int64)):
        with refused("pos.*int32"):
            rows(pos=bad)
    with refused("channels a head"):
        rows(k=z(8, 2, 128), ko=z(8, 2, 128))
    with refused("channels a head"):
        append(q=z(8, 4, 128), qo=z(8, 4, 128))
    for bad in (dict(k=z(8, 3, 64)), dict(v=z(7, 2, 64)), dict(k=z(8, 4, 64)[:, :2])):
        with refused("needed|differ"):
            append(**bad)
    with refused("bfloat16"):
        append(v=z(8, 2, 64, dtype=torch.float16))
    with refused("too short for 3"):
        append(batch=3)


def test_binding_verify(lib):
    c = chunk_of()
    f = lambda *s: torch.zeros(*s)                                             # noqa: E731

    def call(p=f(8, 50), q=f(8, 50), tok=i32(8), au=f(8), su=f(2), c=c, batch=2, na=i32(2), nt=i32(2),
             kp=i32(2)):
        binding.se_draft_verify(p, q, tok, au, su, c, batch, na, nt, kp, WS, stream=NoStream)
    for good in (dict(), dict(q=None), dict(p=f(8, 64)[:, :50], q=f(8, 64)[:, :50])):
        with refused("current CUDA device"):
            call(**good)
    for bad in (dict(p=f(8, 50).double()), dict(p=f(8, 50).half(), q=None), dict(q=f(8, 50).bfloat16()),
                dict(p=f(7, 50)), dict(q=f(7, 50)), dict(q=f(8, 51)), dict(p=f(50, 8).t()),
                dict(q=f(8, 64)[:, :50]), dict(p=f(1, 50).expand(8, 50)), dict(p=f(8, 1, 50), q=None)):
        with refused("probabilities"):
            call(**bad)
    for bad in (dict(tok=i32(7)), dict(tok=i32(8).long()), dict(na=i32(1)), dict(nt=i32(4)[::2]),
                dict(kp=i32(2).long())):
        with refused("int32"):
            call(**bad)
    for bad in (dict(au=f(7)), dict(au=f(8).double()), dict(su=f(1)), dict(su=f(4)[::2])):
        with refused("float32"):
            call(**bad)
    with refused("too short for 3"):
        call(batch=3, su=f(3), na=i32(3), nt=i32(3), kp=i32(3))


def test_binding_tables(lib):
    def args(call, pool=None, refs=i32(6), words=i32(2), batch=2, c=None):
        call(pool or pool_of(), refs, words, batch, c or binding.Carry.empty(2, "cpu"), WS,
             stream=NoStream)
    for call in (binding.se_pages_fork, binding.se_pages_truncate):
        with refused("current CUDA device"):
            args(call)
        for bad in (dict(refs=i32(5)), dict(refs=i32(6).long()), dict(words=i32(1)),
                    dict(words=i32(4)[::2]), dict(words=torch.zeros(2, dtype=torch.bool))):
            with refused("int32"):
                args(call, **bad)
        with refused("Carry.*too short for 2"):
            args(call, c=binding.Carry.empty(1, "cpu"))
        with refused("Carry.from_page.*int32"):
            args(call, c=binding.Carry(i32(2), i32(2).long()))
        with refused("PagePool.*too short for 2"):
            args(call, pool=pool_of(n_pages=i32(1)))
    with refused("current CUDA device"):
        binding.se_pages_carry(cache_of(), binding.Carry.empty(2, "cpu"), 2, WS, stream=NoStream)
    with refused("Carry.*too short for 2"):
        binding.se_pages_carry(cache_of(), binding.Carry.empty(1, "cpu"), 2, WS, stream=NoStream)
    with refused("PagedKV.*too short for 3"):
        binding.se_pages_carry(cache_of(), binding.Carry.empty(3, "cpu"), 3, WS, stream=NoStream)
