"""Thin ctypes binding of libsparse_engine.so (argument marshalling only).

Every function here has the name of the C entry point it calls, takes torch
CUDA tensors, passes their device pointers and the current CUDA stream, and
raises ``SparseEngineError`` on a negative status.  All computation happens in
the library's kernels; there is no Python or CPU fallback: if the library is
not built, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch

from . import build as _build

c_i32p = ctypes.c_void_p  # device pointers are passed as raw addresses


class SparseEngineError(RuntimeError):
    pass


class PagedKVC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class ViewC(ctypes.Structure):
    _fields_ = [("chunk_row", ctypes.c_void_p), ("n_tokens", ctypes.c_void_p),
                ("num_units", ctypes.c_int32), ("max_chunks", ctypes.c_int32)]


class VarlenKVC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("score", ctypes.c_void_p), ("seg_off", ctypes.c_void_p),
                ("seg_len", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("seg_cap", ctypes.c_int32), ("total_rows", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class H2OStateC(ctypes.Structure):
    _fields_ = [("kv", VarlenKVC), ("budget", ctypes.c_int32), ("recent", ctypes.c_int32)]


class PagePoolC(ctypes.Structure):
    _fields_ = [("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_void_p),
                ("n_pages", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("ctx_len", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32)]


class ChunkC(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p), ("seq", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("slot", ctypes.c_void_p), ("max_tokens", ctypes.c_int32)]


class ChunkAttnOptsC(ctypes.Structure):
    _fields_ = [("out_dtype", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sink", ctypes.c_int32), ("q_stride", ctypes.c_int64),
                ("ev_kernel_begin", ctypes.c_void_p), ("ev_kernel_end", ctypes.c_void_p),
                ("wait_limit_ns", ctypes.c_int32)]


class RopeC(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("amplitude", ctypes.c_float), ("eps", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


class RopeScalingC(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_float),
                ("original_len", ctypes.c_float), ("low", ctypes.c_float),
                ("high", ctypes.c_float)]


class PageCarryC(ctypes.Structure):
    _fields_ = [("from_seq", ctypes.c_void_p), ("from_page", ctypes.c_void_p)]


class DecodeOptsC(ctypes.Structure):
    _fields_ = [("out_dtype", ctypes.c_int32), ("max_splits", ctypes.c_int32),
                ("logits_out", ctypes.c_void_p), ("logits_stride", ctypes.c_int32),
                ("ev_kernel_begin", ctypes.c_void_p), ("ev_kernel_end", ctypes.c_void_p)]


class SelectOptsC(ctypes.Structure):
    _fields_ = [("group_agg", ctypes.c_int32)]


SE_AGG_SUM, SE_AGG_MAX = 0, 1
SE_ROPE_HALVES, SE_ROPE_PAIRS = 0, 1
SE_ROPE_PLAIN, SE_ROPE_LINEAR, SE_ROPE_NTK, SE_ROPE_YARN, SE_ROPE_BANDS = range(5)


class QuestStepOptsC(ctypes.Structure):
    _fields_ = [("out_dtype", ctypes.c_int32), ("max_splits", ctypes.c_int32),
                ("ev_kernel_begin", ctypes.c_void_p), ("ev_kernel_end", ctypes.c_void_p),
                ("wait_limit_ns", ctypes.c_int32)]


# C entry points: name -> (restype, argtypes)
_VP, _I, _SZ, _F, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
_F64 = ctypes.c_double
SIGNATURES = {
    "se_status_str": (ctypes.c_char_p, [_I]),
    "se_version": (_I, []),
    "se_sync_status": (_I, [_VP, _VP]),
    "se_small_workspace": (_SZ, []),
    "se_quest_select_workspace": (_SZ, [_I, _I, _I]),
    "se_sparse_decode_workspace": (_SZ, [_I, _I, _I, _I]),
    "se_quest_step_workspace": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "se_snapkv_workspace": (_SZ, [_I, _I, _I, _I, _I]),
    "se_h2o_workspace": (_SZ, [_I, _I, _I, _I, _I]),
    "se_page_pool_workspace": (_SZ, [_I]),
    "se_chunk_attn_workspace": (_SZ, [_I, _I, _I, _I, _I]),
    "se_chunk_plan": (_I, [_VP, _VP, _I, _VP, _VP, _SZ, _VP]),
    "se_pages_release": (_I, [_VP, _VP, _I, _VP, _SZ, _VP]),
    "se_kv_append_chunk": (_I, [_VP, _VP, _VP, _I64, _VP, _I, _VP, _SZ, _VP]),
    "se_chunk_attn": (_I, [_VP, _VP, _VP, _I, _I, _F, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "se_rope_turns": (_I, [_F64, _I, _VP, _VP, _VP]),
    "se_qk_rope": (_I, [_VP, _VP, _I, _I, _I, _I, _VP, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _VP,
                        _SZ, _VP]),
    "se_rope_append_chunk": (_I, [_VP, _VP, _VP, _I64, _I, _VP, _VP, _I64, _VP, _I64, _VP, _I, _VP,
                                  _SZ, _VP]),
    "se_draft_verify_workspace": (_SZ, [_I, _I]),
    "se_draft_verify": (_I, [_VP, _VP, _I64, _I, _I, _VP, _VP, _VP, _VP, _I, _VP, _VP, _VP, _VP,
                             _SZ, _VP]),
    "se_pages_truncate_workspace": (_SZ, [_I, _I]),
    "se_pages_fork": (_I, [_VP, _VP, _VP, _I, _VP, _VP, _SZ, _VP]),
    "se_pages_truncate": (_I, [_VP, _VP, _VP, _I, _VP, _VP, _SZ, _VP]),
    "se_pages_carry": (_I, [_VP, _VP, _I, _VP, _SZ, _VP]),
    "se_page_meta_build": (_I, [_VP, _I, _VP, _SZ, _VP]),
    "se_kv_append": (_I, [_VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "se_quest_select": (_I, [_VP, _VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "se_quest_select_append": (_I, [_VP, _VP, _VP, _VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ,
                                    _VP]),
    "se_quest_step": (_I, [_VP, _VP, _VP, _VP, _I, _I, _VP, _F, _VP, _VP, _VP, _VP, _VP, _VP,
                           _VP, _SZ, _VP]),
    "se_view_from_segments": (_I, [_VP, _I, _VP, _VP, _SZ, _VP]),
    "se_quest_select_ex": (_I, [_VP, _VP, _VP, _VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _SZ,
                                _VP]),
    "se_sparse_decode": (_I, [_VP, _VP, _I64, _VP, _VP, _I, _I, _I, _I, _F, _VP, _VP, _VP,
                              _VP, _SZ, _VP]),
    "se_sparse_decode_noalloc": (_I, [_VP, _VP, _I64, _VP, _VP, _I, _I, _I, _I, _F, _I, _VP,
                                      _VP, _VP, _VP]),
    "se_varlen_append": (_I, [_VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "se_varlen_append_view": (_I, [_VP, _VP, _VP, _I, _VP, _VP, _SZ, _VP]),
    "se_snapkv_compact": (_I, [_VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _VP, _SZ, _VP]),
    "se_h2o_step": (_I, [_VP, _VP, _VP, _VP, _I, _I, _F, _I, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "se_chain_snapshot_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "se_chain_save": (_I, [_VP, _VP, _I, _I, _VP, _SZ, _VP, _SZ, _VP]),
    "se_chain_restore": (_I, [_VP, _SZ, _I, _I, _VP, _VP, _VP, _SZ, _VP]),
    "se_chain_index_create": (_VP, []),
    "se_chain_index_destroy": (None, [_VP]),
    "se_chain_index_put": (_I, [_VP, _VP, _I64, _I64]),
    "se_chain_index_match": (_I64, [_VP, _VP, _I64, _VP]),
    "se_chain_index_erase": (_I, [_VP, _I64]),
    "se_chain_index_size": (_I64, [_VP]),
    "se_span_prune": (_I, [_VP, _VP, _I, _I, _I, _I, _VP, _VP, _F, _VP, _VP, _SZ, _VP]),
    "se_view_sink_recent": (_I, [_VP, _I, _I, _I, _VP, _VP, _SZ, _VP]),
}

_lib = None
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise SparseEngineError(
            f"{path} is missing: build it first (kv_cache_decode_quest_gb300.build.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load().se_status_str(rc).decode()
        raise SparseEngineError(f"{what} failed: {msg} ({rc})")


def _p(t):
    return None if t is None else t.data_ptr()


# The current stream's handle alone (building the torch.cuda.Stream object costs as much as a
# launch).  The function is private to torch: where it is missing, the object is built.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _ref(x):
    return ctypes.byref(x) if x is not None else None


# ---------------------------------------------------------------------------
# holders: keep the tensors alive next to the C struct that points at them
# ---------------------------------------------------------------------------

class _Measured:
    """A holder of tensors whose types and lengths the calls on chunks look at once after each
    assignment, not in every call (`_measure`: the sequences it holds, or an error)."""

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__["_sequences"] = self.__dict__["_device"] = None


def _int32_fields(holder):
    # the kernels take bare pointers: another type would be read as pairs or quarters of words
    for f in dataclasses.fields(holder):
        t = getattr(holder, f.name)
        if t.dtype is not torch.int32 or not t.is_contiguous():
            raise SparseEngineError(f"{type(holder).__name__}.{f.name}: contiguous int32 tensor "
                                    f"needed, got {t.dtype}, strides {t.stride()}")


def _holds(holder: _Measured, batch: int, what: str):
    n = holder._sequences
    if n is None:
        n = holder.__dict__["_sequences"] = holder._measure()
    if n < batch:
        raise SparseEngineError(f"{what}: the {type(holder).__name__}'s tensors are too short for "
                                f"{batch} sequences")


def _summarises(kv, batch: int, what: str):
    """_holds, and room for the page summaries of `batch` sequences (or none kept)."""
    _holds(kv, batch, what)
    if kv._summarised < batch:
        raise SparseEngineError(f"{what}: contiguous PagedKV.meta of at least [{batch}][max_pages][heads][2]"
                                f"[head_dim] needed, got {tuple(kv.meta.shape)}")


@dataclasses.dataclass
class PagedKV(_Measured):
    k: torch.Tensor            # bf16 [num_pages][Hkv][16][D]
    v: torch.Tensor
    meta: torch.Tensor         # bf16 [B][max_pages][Hkv][2][D], logical page order
    block_table: torch.Tensor  # int32 [B][max_pages]
    ctx_len: torch.Tensor      # int32 [B]

    def _measure(self) -> int:
        k, v, meta, table = self.k, self.v, self.meta, self.block_table
        for t in (k, v, meta):
            if t is not None and t.dtype is not torch.bfloat16:
                raise SparseEngineError(f"PagedKV: a bfloat16 cache is needed, got {t.dtype}")
        if k.dim() != 4 or k.shape != v.shape or not k.is_contiguous() or not v.is_contiguous():
            raise SparseEngineError("PagedKV: contiguous k and v of one shape [pages][heads][16][head_dim] "
                                    f"needed, got {tuple(k.shape)} and {tuple(v.shape)}")
        for t, dims, name in ((table, 2, "block_table"), (self.ctx_len, 1, "ctx_len")):
            if t.dtype is not torch.int32 or t.dim() != dims or not t.is_contiguous():
                raise SparseEngineError(f"PagedKV.{name}: contiguous int32 tensor of {dims} dimension(s) "
                                        f"needed, got {t.dtype} of shape {tuple(t.shape)}")
        n = min(self.ctx_len.numel(), table.shape[0])
        # sequences whose summaries may be written (a call that only reads pages takes any)
        fits = meta is None or (meta.is_contiguous() and
                                meta.shape[1:] == (table.shape[1], k.shape[1], 2, k.shape[3]))
        self.__dict__["_summarised"] = n if meta is None else min(n, meta.shape[0]) if fits else -1
        return n

    @property
    def c(self) -> PagedKVC:
        k, meta, table = self.k, self.meta, self.block_table
        P, H, S, D = k.shape
        return PagedKVC(k.data_ptr(), self.v.data_ptr(), None if meta is None else meta.data_ptr(),
                        table.data_ptr(), self.ctx_len.data_ptr(), P, table.shape[1], H, D, S)


@dataclasses.dataclass
class View:
    chunk_row: torch.Tensor    # int32 [units][max_chunks]
    n_tokens: torch.Tensor     # int32 [units]

    @property
    def c(self) -> ViewC:
        return ViewC(_p(self.chunk_row), _p(self.n_tokens), self.chunk_row.shape[0],
                     self.chunk_row.shape[1])

    @staticmethod
    def empty(units: int, max_chunks: int, device="cuda") -> "View":
        return View(torch.zeros(units, max_chunks, dtype=torch.int32, device=device),
                    torch.zeros(units, dtype=torch.int32, device=device))


@dataclasses.dataclass
class VarlenKV:
    k: torch.Tensor            # bf16 [rows][D]
    v: torch.Tensor
    pos: torch.Tensor          # int32 [rows]
    score: torch.Tensor | None # fp32 [rows]
    seg_off: torch.Tensor      # int32 [units]
    seg_len: torch.Tensor      # int32 [units]
    seq_len: torch.Tensor      # int32 [B]
    seg_cap: int
    num_kv_heads: int

    @property
    def c(self) -> VarlenKVC:
        return VarlenKVC(_p(self.k), _p(self.v), _p(self.pos), _p(self.score), _p(self.seg_off),
                         _p(self.seg_len), _p(self.seq_len), self.seg_cap, self.k.shape[0],
                         self.num_kv_heads, self.k.shape[1])

    @staticmethod
    def empty(batch: int, num_kv_heads: int, seg_cap: int, head_dim: int, with_score=False,
              device="cuda") -> "VarlenKV":
        units = batch * num_kv_heads
        rows = units * seg_cap
        return VarlenKV(
            torch.zeros(rows, head_dim, dtype=torch.bfloat16, device=device),
            torch.zeros(rows, head_dim, dtype=torch.bfloat16, device=device),
            torch.full((rows,), -1, dtype=torch.int32, device=device),
            torch.zeros(rows, dtype=torch.float32, device=device) if with_score else None,
            torch.arange(units, dtype=torch.int32, device=device) * seg_cap,
            torch.zeros(units, dtype=torch.int32, device=device),
            torch.zeros(batch, dtype=torch.int32, device=device),
            seg_cap, num_kv_heads)


@dataclasses.dataclass
class H2OState:
    kv: VarlenKV               # with score
    budget: int
    recent: int

    @property
    def c(self) -> H2OStateC:
        return H2OStateC(self.kv.c, self.budget, self.recent)


@dataclasses.dataclass
class PagePool(_Measured):
    free_pages: torch.Tensor   # int32 [num_pages], the first n_free entries are free
    n_free: torch.Tensor       # int32 [1]
    n_pages: torch.Tensor      # int32 [B]
    block_table: torch.Tensor  # int32 [B][max_pages], the PagedKV's
    ctx_len: torch.Tensor      # int32 [B], the PagedKV's

    def _measure(self) -> int:
        _int32_fields(self)
        if self.n_free.numel() < 1:
            raise SparseEngineError("PagePool.n_free: one word needed")
        return min(self.n_pages.numel(), self.ctx_len.numel(), self.block_table.shape[0])

    @property
    def c(self) -> PagePoolC:
        return PagePoolC(self.free_pages.data_ptr(), self.n_free.data_ptr(),
                         self.n_pages.data_ptr(), self.block_table.data_ptr(),
                         self.ctx_len.data_ptr(), self.free_pages.numel(),
                         self.block_table.shape[1])

    @staticmethod
    def empty(batch: int, num_pages: int, max_pages_per_seq: int, device="cuda") -> "PagePool":
        """Every page free (page 0 handed out first), no sequence holds any."""
        return PagePool(
            torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
            torch.full((1,), num_pages, dtype=torch.int32, device=device),
            torch.zeros(batch, dtype=torch.int32, device=device),
            torch.full((batch, max_pages_per_seq), -1, dtype=torch.int32, device=device),
            torch.zeros(batch, dtype=torch.int32, device=device))


@dataclasses.dataclass
class Chunk(_Measured):
    start: torch.Tensor        # int32 [B + 1]
    seq: torch.Tensor          # int32 [max_tokens]
    pos: torch.Tensor          # int32 [max_tokens]
    slot: torch.Tensor         # int32 [max_tokens]

    def _measure(self) -> int:
        _int32_fields(self)
        if min(self.pos.numel(), self.slot.numel()) < self.seq.numel():
            raise SparseEngineError("Chunk: fewer entries in pos or slot than rows in seq")
        return self.start.numel() - 1

    @property
    def c(self) -> ChunkC:
        return ChunkC(self.start.data_ptr(), self.seq.data_ptr(), self.pos.data_ptr(),
                      self.slot.data_ptr(), self.seq.numel())

    @staticmethod
    def empty(batch: int, max_tokens: int, device="cuda") -> "Chunk":
        rows = torch.full((3, max_tokens), -1, dtype=torch.int32, device=device)
        return Chunk(torch.zeros(batch + 1, dtype=torch.int32, device=device), rows[0], rows[1],
                     rows[2])


@dataclasses.dataclass
class Carry(_Measured):
    """What each layer's cache takes over after se_pages_fork or se_pages_truncate."""
    from_seq: torch.Tensor     # int32 [B]
    from_page: torch.Tensor    # int32 [B]

    def _measure(self) -> int:
        _int32_fields(self)
        return min(self.from_seq.numel(), self.from_page.numel())

    @property
    def c(self) -> PageCarryC:
        return PageCarryC(self.from_seq.data_ptr(), self.from_page.data_ptr())

    @staticmethod
    def empty(batch: int, device="cuda") -> "Carry":
        t = torch.full((2, batch), -1, dtype=torch.int32, device=device)
        return Carry(t[0], t[1])


@dataclasses.dataclass
class Rope(_Measured):
    """A layer's rotation and the norms ahead of it (Rope.make)."""
    turns: torch.Tensor | None           # int64 [rot_dim / 2], the 64 bits of turns per position
    rot_dim: int
    layout: int = SE_ROPE_HALVES
    amplitude: float = 1.0
    eps: float = 1e-6
    q_weight: torch.Tensor | None = None     # bf16 [D]
    k_weight: torch.Tensor | None = None     # bf16 [D]

    def _measure(self) -> int:
        t = self.turns
        if t is not None and (t.dtype is not torch.int64 or not t.is_contiguous()):
            raise SparseEngineError(f"Rope.turns: contiguous int64 tensor needed, got {t.dtype}")
        if self.rot_dim and (t is None or 2 * t.numel() < self.rot_dim):
            raise SparseEngineError(f"Rope.turns: {self.rot_dim // 2} entries needed")
        widths = set()
        for name in ("q_weight", "k_weight"):
            w = getattr(self, name)
            if w is not None:
                if w.dtype is not _BF16 or not w.is_contiguous() or w.dim() != 1:
                    raise SparseEngineError(f"Rope.{name}: contiguous bfloat16 [head_dim] needed, got "
                                            f"{w.dtype} of shape {tuple(w.shape)}")
                widths.add(w.numel())
        if len(widths) > 1:
            raise SparseEngineError("Rope: norm weights of two lengths")
        return widths.pop() if widths else 0

    @property
    def c(self) -> RopeC:
        t, q, k = self.turns, self.q_weight, self.k_weight
        return RopeC(None if t is None else t.data_ptr(), self.rot_dim, self.layout, self.amplitude,
                     self.eps, None if q is None else q.data_ptr(),
                     None if k is None else k.data_ptr())

    @staticmethod
    def make(rot_dim: int, base: float = 10000.0, scaling: int = SE_ROPE_PLAIN, factor: float = 1.0,
             original_len: float = 0.0, low: float = 1.0, high: float = 32.0,
             layout: int = SE_ROPE_HALVES, q_weight=None, k_weight=None, eps: float = 1e-6,
             amplitude: float | None = None, device="cuda") -> "Rope":
        """The rotation of rot_dim channels (0: norms alone); amplitude None: the scaling's own."""
        turns, amp = None, 1.0
        if rot_dim:
            turns, amp = se_rope_turns(rot_dim, base, scaling, factor, original_len, low, high)
            turns = turns.to(device)
        return Rope(turns, rot_dim, layout, amp if amplitude is None else amplitude, eps, q_weight,
                    k_weight)


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zeroed device workspace (status word cleared)."""
    return torch.zeros(max(256, int(nbytes)), dtype=torch.uint8, device=device)


def se_sync_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the SE_DEV_* bits of the workspace's
    status word (raises on a negative status)."""
    rc = load().se_sync_status(_p(ws), _stream(stream))
    if rc < 0:
        _check(rc, "se_sync_status")
    return rc


def status_word(ws: torch.Tensor) -> int:
    """The device status word of a workspace, read through se_sync_status."""
    return se_sync_status(ws)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def se_version() -> int:
    return load().se_version()


def se_small_workspace() -> int:
    return load().se_small_workspace()


def se_quest_select_workspace(batch, num_kv_heads, max_pages_per_seq) -> int:
    return load().se_quest_select_workspace(batch, num_kv_heads, max_pages_per_seq)


def se_sparse_decode_workspace(num_units, group_size, head_dim, max_splits=64) -> int:
    return load().se_sparse_decode_workspace(num_units, group_size, head_dim, max_splits)


def se_quest_step_workspace(batch, num_kv_heads, num_q_heads, head_dim, max_pages_per_seq,
                            max_splits=64) -> int:
    return load().se_quest_step_workspace(batch, num_kv_heads, num_q_heads, head_dim,
                                          max_pages_per_seq, max_splits)


def se_snapkv_workspace(batch, num_kv_heads, num_q_heads, window, max_ctx) -> int:
    return load().se_snapkv_workspace(batch, num_kv_heads, num_q_heads, window, max_ctx)


def se_h2o_workspace(batch, num_kv_heads, num_q_heads, head_dim, seg_cap) -> int:
    return load().se_h2o_workspace(batch, num_kv_heads, num_q_heads, head_dim, seg_cap)


def se_page_meta_build(kv: PagedKV, batch: int, ws, stream=None):
    c = kv.c
    _check(load().se_page_meta_build(ctypes.byref(c), batch, _p(ws), ws.numel(), _stream(stream)),
           "se_page_meta_build")


def se_kv_append(kv: PagedKV, k_new, v_new, batch: int, ws, stream=None):
    c = kv.c
    _check(load().se_kv_append(ctypes.byref(c), _p(k_new), _p(v_new), batch, _p(ws), ws.numel(),
                               _stream(stream)), "se_kv_append")


def se_page_pool_workspace(batch: int) -> int:
    return load().se_page_pool_workspace(batch)


def se_chunk_attn_workspace(batch, max_tokens, num_kv_heads, num_q_heads, head_dim) -> int:
    return load().se_chunk_attn_workspace(batch, max_tokens, num_kv_heads, num_q_heads, head_dim)


def _per_sequence(t, batch: int, what: str):
    """An int32 word for each of `batch` sequences (None: the library's check)."""
    if t is not None and (t.dtype is not _I32 or t.numel() < batch or not t.is_contiguous()):
        raise SparseEngineError(f"{what}: contiguous int32 of at least {batch} entries needed, got "
                                f"{t.dtype} of shape {tuple(t.shape)}")


def se_chunk_plan(pool: PagePool, new_len, batch: int, chunk: Chunk, ws, stream=None):
    """Pages, positions and cache rows of each sequence's new tokens."""
    c, cc = pool.c, chunk.c
    _per_sequence(new_len, batch, "se_chunk_plan new_len")
    _holds(pool, batch, "se_chunk_plan")
    _holds(chunk, batch, "se_chunk_plan")
    _check(load().se_chunk_plan(ctypes.byref(c), _p(new_len), batch, ctypes.byref(cc), _p(ws),
                                ws.numel(), _stream(stream)), "se_chunk_plan")


def se_pages_release(pool: PagePool, done, batch: int, ws, stream=None):
    """Pages of the sequences with done[b] != 0 back onto the free stack."""
    c = pool.c
    _per_sequence(done, batch, "se_pages_release done")
    _holds(pool, batch, "se_pages_release")
    _check(load().se_pages_release(ctypes.byref(c), _p(done), batch, _p(ws), ws.numel(),
                                   _stream(stream)), "se_pages_release")


def _token_stride(x, what: str, tokens: int = 0, heads: int = 0, head_dim: int = 0):
    """Elements between tokens of a [tokens][heads][head_dim] tensor, which may be a
    slice of wider rows (a packed q/k/v projection).  With `heads` the shape is checked too:
    the kernels reach every row up to the chunk's max_tokens."""
    shape, stride = x.shape, x.stride()
    try:
        n, h, d = shape
        sn, sh, sd = stride
        ok = n == 0 or sd == 1 and (sh == d or h == 1)     # (no rows: strides mean nothing)
    except ValueError:
        ok = False
    if not ok:
        raise SparseEngineError(f"{what}: [tokens][heads][head_dim] with contiguous heads needed, "
                                f"got shape {tuple(shape)} strides {stride}")
    if heads and (h != heads or d != head_dim or n < tokens):
        raise SparseEngineError(f"{what}: shape {tuple(shape)}, needed is at least "
                                f"[{tokens}][{heads}][{head_dim}]")
    if n <= 1:
        return h * d
    if sn < h * d:
        raise SparseEngineError(f"{what}: tokens overlap (an expanded tensor?), strides {stride}")
    return sn


def se_kv_append_chunk(kv: PagedKV, k_new, v_new, chunk: Chunk, batch: int, ws, stream=None):
    """Append the chunk's rows; k_new and v_new [max_tokens][Hkv][D] may be slices
    of wider rows."""
    c, cc = kv.c, chunk.c
    rows, heads, dim = cc.max_tokens, c.num_kv_heads, c.head_dim
    stride = _token_stride(k_new, "se_kv_append_chunk k_new", rows, heads, dim)
    if stride != _token_stride(v_new, "se_kv_append_chunk v_new", rows, heads, dim):
        raise SparseEngineError("se_kv_append_chunk: k_new and v_new strides differ")
    if k_new.dtype is not _BF16 or v_new.dtype is not _BF16:
        raise SparseEngineError("se_kv_append_chunk: bfloat16 k_new and v_new needed")
    _summarises(kv, batch, "se_kv_append_chunk")
    _holds(chunk, 0, "se_kv_append_chunk")
    _check(load().se_kv_append_chunk(ctypes.byref(c), _p(k_new), _p(v_new), stride,
                                     ctypes.byref(cc), batch, _p(ws), ws.numel(),
                                     _stream(stream)), "se_kv_append_chunk")


def se_chunk_attn(kv: PagedKV, q, chunk: Chunk, batch: int, num_q_heads: int, scale: float, out,
                  lse, ws, out_dtype: int = 0, window: int = 0, sink: int = 0, ev_begin=None,
                  ev_end=None, stream=None, wait_limit_ns: int = 0):
    """Causal attention of the chunk's tokens over the paged cache; q
    [max_tokens][Hq][D] may be a slice of wider rows."""
    c, cc = kv.c, chunk.c
    rows, dim = cc.max_tokens, c.head_dim
    stride = _token_stride(q, "se_chunk_attn q", rows, num_q_heads, dim)
    _token_stride(out, "se_chunk_attn out", rows, num_q_heads, dim)
    if q.dtype is not _BF16:
        raise SparseEngineError("se_chunk_attn: bfloat16 q needed")
    if not out.is_contiguous() or out.dtype is not (_F32 if out_dtype else _BF16):
        raise SparseEngineError("se_chunk_attn: out is not contiguous or not of out_dtype")
    if lse is not None and (lse.numel() < rows * num_q_heads or not lse.is_contiguous() or
                            lse.dtype is not _F32):
        raise SparseEngineError("se_chunk_attn: float32 lse of [max_tokens][num_q_heads] needed")
    _holds(kv, batch, "se_chunk_attn")
    _holds(chunk, batch, "se_chunk_attn")
    opts = ChunkAttnOptsC(out_dtype, window, sink, stride,
                          ev_begin.cuda_event if ev_begin is not None else None,
                          ev_end.cuda_event if ev_end is not None else None, wait_limit_ns)
    _check(load().se_chunk_attn(ctypes.byref(c), _p(q), ctypes.byref(cc), batch, num_q_heads,
                                scale, ctypes.byref(opts), _p(out), _p(lse), _p(ws), ws.numel(),
                                _stream(stream)), "se_chunk_attn")


# the current device's number alone (private to torch, as above)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _elsewhere(what: str, device: int):
    where = "the CPU or several devices" if device < 0 else f"cuda:{device}"
    raise SparseEngineError(f"{what}: a tensor is on {where}, not on the current CUDA device")


def _located(holder: _Measured) -> int:
    """The one device of a holder's tensors (-1: the CPU, -2: several), looked up once after each
    assignment."""
    found = {t.get_device() for f in dataclasses.fields(holder)
             if isinstance(t := getattr(holder, f.name), torch.Tensor)}
    at = holder.__dict__["_device"] = found.pop() if len(found) == 1 else -2 if found else -3
    return at


def _on_device(what: str, holders, *tensors) -> int:
    """The current device; refuses tensors that its kernels cannot reach."""
    here = tensors[0].get_device()
    if here < 0 or here != _current_device():
        _elsewhere(what, here)
    for t in tensors[1:]:
        if t is not None and t.get_device() != here:
            _elsewhere(what, t.get_device())
    for h in holders:
        at = h._device
        if at is None:
            at = _located(h)
        if at != here and at != -3:                    # (-3: it holds no tensor)
            _elsewhere(what, at)
    return here


def _stream_on(device: int, stream):
    if stream is not None or _raw_stream is None:
        return _stream(stream)
    return _raw_stream(device)


def se_rope_turns(rot_dim: int, base: float = 10000.0, scaling: int = SE_ROPE_PLAIN,
                  factor: float = 1.0, original_len: float = 0.0, low: float = 1.0,
                  high: float = 32.0):
    """(turns, amplitude): the frequencies of a rotation as int64 (CPU) and the factor on its cosines."""
    turns = torch.zeros(max(0, rot_dim // 2), dtype=torch.int64)
    amplitude = ctypes.c_float(1.0)
    s = RopeScalingC(scaling, factor, original_len, low, high)
    _check(load().se_rope_turns(base, rot_dim, ctypes.byref(s), _p(turns), ctypes.byref(amplitude)),
           "se_rope_turns")
    return turns, amplitude.value


def _rope_fits(rope: Rope, dim: int, what: str):
    n = rope._sequences
    if n is None:
        n = rope.__dict__["_sequences"] = rope._measure()
    if n and n != dim:
        raise SparseEngineError(f"{what}: norm weights of {n} channels, heads of {dim}")


def _rotated(x, out, rows: int, what: str):
    """(heads, head_dim, stride, out stride) of rows of heads and the tensor they go to."""
    if x is None or out is None:
        if x is not out:
            raise SparseEngineError(f"{what}: rows without a tensor to go to, or the other way round")
        return 0, 0, 0, 0
    if x.dtype is not _BF16 or out.dtype is not _BF16:
        raise SparseEngineError(f"{what}: bfloat16 needed, got {x.dtype} and {out.dtype}")
    shape, stride = x.shape, x.stride()
    to = stride if out is x else out.stride()
    if len(shape) == 3 == len(to) and rows > 1:            # the usual rows at one look
        n, h, d = shape
        if stride[2] == 1 == to[2] and stride[1] == d == to[1] and n >= rows and \
                stride[0] >= h * d <= to[0] and out.shape == shape:
            return h, d, stride[0], to[0]
    if len(shape) != 3:
        shape = rows, 0, 0                                 # (refused below)
    return (shape[1], shape[2], _token_stride(x, what, rows, shape[1], shape[2]),
            _token_stride(out, what + "_out", rows, shape[1], shape[2]))


def se_qk_rope(rope: Rope, pos, q, k, q_out, k_out, ws, stream=None):
    """Queries [rows][Hq][D] and keys [rows][Hkv][D] (or one of them, the other None) normalised per
    head and rotated to the positions pos (int32 [rows], negative: the row is left out); q_out may be q
    and k_out k, and all may be slices of wider rows."""
    rows = pos.numel()
    _per_sequence(pos, rows, "se_qk_rope pos")
    hq, dim, sq, oq = _rotated(q, q_out, rows, "se_qk_rope q")
    hk, dim_k, sk, ok = _rotated(k, k_out, rows, "se_qk_rope k")
    if hq and hk and dim != dim_k:
        raise SparseEngineError(f"se_qk_rope: q of {dim} channels a head, k of {dim_k}")
    dim = dim or dim_k
    _rope_fits(rope, dim, "se_qk_rope")
    here = _on_device("se_qk_rope", (rope,), pos, ws, q, k, q_out, k_out)
    c = rope.c
    rc = load().se_qk_rope(ctypes.byref(c), pos.data_ptr(), rows, hq, hk, dim, _p(q), sq, _p(k), sk,
                           _p(q_out), oq, _p(k_out), ok, ws.data_ptr(), ws.numel(),
                           _stream_on(here, stream))
    if rc:
        _check(rc, "se_qk_rope")


def se_rope_append_chunk(kv: PagedKV, rope: Rope, q, k_new, v_new, q_out, chunk: Chunk, batch: int,
                         ws, stream=None):
    """se_qk_rope of the chunk's rows and se_kv_append_chunk of the rotated keys and of v_new in one
    pass; q, q_out None: keys alone.  All rows may be slices of wider rows."""
    c, cc = kv.c, chunk.c
    rows, heads, dim = cc.max_tokens, c.num_kv_heads, c.head_dim
    stride = _token_stride(k_new, "se_rope_append_chunk k_new", rows, heads, dim)
    if stride != _token_stride(v_new, "se_rope_append_chunk v_new", rows, heads, dim):
        raise SparseEngineError("se_rope_append_chunk: k_new and v_new strides differ")
    if k_new.dtype is not _BF16 or v_new.dtype is not _BF16:
        raise SparseEngineError("se_rope_append_chunk: bfloat16 k_new and v_new needed")
    hq, dim_q, sq, oq = _rotated(q, q_out, rows, "se_rope_append_chunk q")
    if hq and dim_q != dim:
        raise SparseEngineError(f"se_rope_append_chunk: q of {dim_q} channels a head, the cache of {dim}")
    _rope_fits(rope, dim, "se_rope_append_chunk")
    _summarises(kv, batch, "se_rope_append_chunk")
    _holds(chunk, 0, "se_rope_append_chunk")
    here = _on_device("se_rope_append_chunk", (kv, rope, chunk), k_new, v_new, ws, q, q_out)
    rc = rope.c
    rc = load().se_rope_append_chunk(ctypes.byref(c), ctypes.byref(rc), _p(q), sq, hq,
                                     k_new.data_ptr(), v_new.data_ptr(), stride, _p(q_out), oq,
                                     ctypes.byref(cc), batch, ws.data_ptr(), ws.numel(),
                                     _stream_on(here, stream))
    if rc:
        _check(rc, "se_rope_append_chunk")


def se_draft_verify_workspace(batch: int, vocab: int) -> int:
    return load().se_draft_verify_workspace(batch, vocab)


def se_draft_verify(probs, draft_probs, tokens, accept_u, sample_u, chunk: Chunk, batch: int,
                    n_accepted, next_token, keep, ws, stream=None):
    """Which of the chunk's drafted tokens stay and the token behind them; probs and draft_probs (or
    None) [max_tokens][vocab] bf16 or fp32, keep: the lengths for se_pages_truncate."""
    what, rows = "se_draft_verify", chunk.seq.numel()
    dtype, shape, stride = probs.dtype, probs.shape, probs.stride()
    for t in (probs,) if draft_probs is None else (probs, draft_probs):
        if t.dtype is not dtype or (dtype is not _F32 and dtype is not _BF16):
            raise SparseEngineError(f"{what}: probabilities in bfloat16 or float32 needed, one type for "
                                    f"both, got {t.dtype}")
        at, by = t.shape, t.stride()
        if len(at) != 2 or len(shape) != 2 or at[0] < rows or at[1] != shape[1] or \
                (rows > 0 and at[1] > 1 and by[1] != 1) or \
                (rows > 1 and (by[0] != stride[0] or by[0] < at[1])):
            raise SparseEngineError(f"{what}: probabilities of at least [{rows}][vocab] with equal row "
                                    f"strides needed, got shape {tuple(at)} strides {by}")
    _per_sequence(tokens, rows, f"{what} tokens")
    for t, n, name in ((accept_u, rows, "accept_u"), (sample_u, batch, "sample_u")):
        if t.dtype is not _F32 or t.numel() < n or not t.is_contiguous():
            raise SparseEngineError(f"{what} {name}: contiguous float32 of at least {n} entries needed, "
                                    f"got {t.dtype} of shape {tuple(t.shape)}")
    for t, name in ((n_accepted, "n_accepted"), (next_token, "next_token"), (keep, "keep")):
        _per_sequence(t, batch, f"{what} {name}")
    _holds(chunk, batch, what)
    here = _on_device(what, (chunk,), probs, draft_probs, tokens, accept_u, sample_u, n_accepted,
                      next_token, keep, ws)
    cc, vocab = chunk.c, shape[1]
    rc = load().se_draft_verify(probs.data_ptr(), _p(draft_probs), stride[0] if rows > 1 else vocab,
                                int(dtype is _F32), vocab, tokens.data_ptr(), accept_u.data_ptr(), sample_u.data_ptr(),
                                ctypes.byref(cc), batch, n_accepted.data_ptr(), next_token.data_ptr(),
                                keep.data_ptr(), ws.data_ptr(), ws.numel(), _stream_on(here, stream))
    if rc:
        _check(rc, what)


def se_pages_truncate_workspace(batch: int, num_pages: int) -> int:
    return load().se_pages_truncate_workspace(batch, num_pages)


def _table_edit(name: str, pool: PagePool, page_refs, words, batch: int, carry: Carry, ws, stream):
    _per_sequence(words, batch, name)
    _per_sequence(page_refs, pool.free_pages.numel(), f"{name} page_refs")
    _holds(pool, batch, name)
    _holds(carry, batch, name)
    here = _on_device(name, (pool, carry), words, page_refs, ws)
    c, cc = pool.c, carry.c
    rc = getattr(load(), name)(ctypes.byref(c), _p(page_refs), words.data_ptr(), batch,
                               ctypes.byref(cc), ws.data_ptr(), ws.numel(), _stream_on(here, stream))
    if rc:
        _check(rc, name)


def se_pages_fork(pool: PagePool, page_refs, src, batch: int, carry: Carry, ws, stream=None):
    """Every sequence b with src[b] >= 0 becomes a copy of sequence src[b] that shares its full pages;
    page_refs int32 [num_pages] counts the holders beside the first."""
    _table_edit("se_pages_fork", pool, page_refs, src, batch, carry, ws, stream)


def se_pages_truncate(pool: PagePool, page_refs, keep, batch: int, carry: Carry, ws, stream=None):
    """Cuts every sequence b with keep[b] >= 0 to keep[b] tokens; pages that nobody holds any more go
    back on the stack.  page_refs None: no pages are shared."""
    _table_edit("se_pages_truncate", pool, page_refs, keep, batch, carry, ws, stream)


def se_pages_carry(kv: PagedKV, carry: Carry, batch: int, ws, stream=None):
    """One layer's cache follows a fork or a truncation: last pages' rows and page summaries."""
    _summarises(kv, batch, "se_pages_carry")
    _holds(carry, batch, "se_pages_carry")
    here = _on_device("se_pages_carry", (kv, carry), ws)
    c, cc = kv.c, carry.c
    rc = load().se_pages_carry(ctypes.byref(c), ctypes.byref(cc), batch, ws.data_ptr(), ws.numel(),
                               _stream_on(here, stream))
    if rc:
        _check(rc, "se_pages_carry")


def se_quest_select(kv: PagedKV, q, batch: int, num_q_heads: int, budget_tokens, sel_pages,
                    n_sel, view: View, ws, stream=None):
    c, vc = kv.c, view.c
    _check(load().se_quest_select(ctypes.byref(c), _p(q), batch, num_q_heads, _p(budget_tokens),
                                  _p(sel_pages), _p(n_sel), ctypes.byref(vc), _p(ws), ws.numel(),
                                  _stream(stream)), "se_quest_select")


def se_quest_select_append(kv: PagedKV, k_new, v_new, q, batch: int, num_q_heads: int,
                           budget_tokens, sel_pages, n_sel, view: View, ws, stream=None):
    c, vc = kv.c, view.c
    _check(load().se_quest_select_append(ctypes.byref(c), _p(k_new), _p(v_new), _p(q), batch,
                                         num_q_heads, _p(budget_tokens), _p(sel_pages),
                                         _p(n_sel), ctypes.byref(vc), _p(ws), ws.numel(),
                                         _stream(stream)), "se_quest_select_append")


def se_quest_select_ex(kv: PagedKV, k_new, v_new, q, batch: int, num_q_heads: int,
                       budget_tokens, sel_pages, n_sel, view: View, ws, group_agg: int = 0,
                       stream=None):
    """Quest selection (with the append when k_new/v_new are given) with
    options: group_agg SE_AGG_SUM or SE_AGG_MAX."""
    c, vc = kv.c, view.c
    opts = SelectOptsC(group_agg)
    _check(load().se_quest_select_ex(ctypes.byref(c), _p(k_new), _p(v_new), _p(q), batch,
                                     num_q_heads, _p(budget_tokens), ctypes.byref(opts),
                                     _p(sel_pages), _p(n_sel), ctypes.byref(vc), _p(ws),
                                     ws.numel(), _stream(stream)), "se_quest_select_ex")


def se_quest_step(kv: PagedKV, k_new, v_new, q, batch: int, num_q_heads: int, budget_tokens,
                  scale: float, sel_pages, n_sel, view: View, out, lse, ws, out_dtype: int = 0,
                  max_splits: int = 64, wait_limit_ns: int = 0, ev_begin=None, ev_end=None,
                  stream=None):
    """One Quest decode step (append when k_new/v_new are given, select, decode)
    in one kernel."""
    c, vc = kv.c, view.c
    opts = QuestStepOptsC(out_dtype, max_splits,
                          ev_begin.cuda_event if ev_begin is not None else None,
                          ev_end.cuda_event if ev_end is not None else None,
                          wait_limit_ns)
    _check(load().se_quest_step(ctypes.byref(c), _p(k_new), _p(v_new), _p(q), batch, num_q_heads,
                                _p(budget_tokens), scale, ctypes.byref(opts), _p(sel_pages),
                                _p(n_sel), ctypes.byref(vc), _p(out), _p(lse), _p(ws), ws.numel(),
                                _stream(stream)), "se_quest_step")


def se_view_from_segments(kv: VarlenKV, batch: int, view: View, ws, stream=None):
    c, vc = kv.c, view.c
    _check(load().se_view_from_segments(ctypes.byref(c), batch, ctypes.byref(vc), _p(ws),
                                        ws.numel(), _stream(stream)), "se_view_from_segments")


def se_sparse_decode(k_rows, v_rows, view: View, q, batch: int, num_q_heads: int,
                     num_kv_heads: int, head_dim: int, scale: float, out, lse, ws,
                     out_dtype: int = 0, max_splits: int = 64, logits_out=None,
                     logits_stride: int = 0, ev_begin=None, ev_end=None, stream=None):
    vc = view.c
    opts = DecodeOptsC(out_dtype, max_splits, _p(logits_out), logits_stride,
                       ev_begin.cuda_event if ev_begin is not None else None,
                       ev_end.cuda_event if ev_end is not None else None)
    total_rows = k_rows.numel() // head_dim
    _check(load().se_sparse_decode(_p(k_rows), _p(v_rows), total_rows, ctypes.byref(vc), _p(q),
                                   batch, num_q_heads, num_kv_heads, head_dim, scale,
                                   ctypes.byref(opts), _p(out), _p(lse), _p(ws), ws.numel(),
                                   _stream(stream)), "se_sparse_decode")


def se_sparse_decode_noalloc(k_rows, v_rows, view: View, q, batch: int, num_q_heads: int,
                             num_kv_heads: int, head_dim: int, scale: float, out, lse,
                             out_dtype: int = 0, status_out=None, stream=None):
    """se_sparse_decode without a workspace (scratch inside the library)."""
    vc = view.c
    total_rows = k_rows.numel() // head_dim
    _check(load().se_sparse_decode_noalloc(_p(k_rows), _p(v_rows), total_rows, ctypes.byref(vc),
                                           _p(q), batch, num_q_heads, num_kv_heads, head_dim,
                                           scale, out_dtype, _p(out), _p(lse), _p(status_out),
                                           _stream(stream)), "se_sparse_decode_noalloc")


def se_varlen_append(kv: VarlenKV, k_new, v_new, batch: int, ws, stream=None):
    c = kv.c
    _check(load().se_varlen_append(ctypes.byref(c), _p(k_new), _p(v_new), batch, _p(ws),
                                   ws.numel(), _stream(stream)), "se_varlen_append")


def se_varlen_append_view(kv: VarlenKV, k_new, v_new, batch: int, view: View, ws, stream=None):
    c, vc = kv.c, view.c
    _check(load().se_varlen_append_view(ctypes.byref(c), _p(k_new), _p(v_new), batch,
                                        ctypes.byref(vc), _p(ws), ws.numel(), _stream(stream)),
           "se_varlen_append_view")


def se_snapkv_compact(prefill: PagedKV, q_win, batch: int, num_q_heads: int, window: int,
                      pool_kernel: int, keep: int, recent: int, scale: float, out: VarlenKV, ws,
                      stream=None):
    c, oc = prefill.c, out.c
    _check(load().se_snapkv_compact(ctypes.byref(c), _p(q_win), batch, num_q_heads, window,
                                    pool_kernel, keep, recent, scale, ctypes.byref(oc), _p(ws),
                                    ws.numel(), _stream(stream)), "se_snapkv_compact")


def se_h2o_step(st: H2OState, q, k_new, v_new, batch: int, num_q_heads: int, scale: float,
                out, lse, evicted_pos, ws, out_dtype: int = 0, stream=None):
    c = st.c
    _check(load().se_h2o_step(ctypes.byref(c), _p(q), _p(k_new), _p(v_new), batch, num_q_heads,
                              scale, out_dtype, _p(out), _p(lse), _p(evicted_pos), _p(ws),
                              ws.numel(), _stream(stream)), "se_h2o_step")


def se_span_prune(prefix: PagedKV, q_win, batch: int, num_q_heads: int, window: int,
                  pool_kernel: int, span, keep_tokens, scale: float, out: VarlenKV, ws,
                  stream=None):
    """Prune each sequence's span [span[b,0], span[b,1]) to its best
    keep_tokens[b] tokens by window score; everything else is kept."""
    c, oc = prefix.c, out.c
    _check(load().se_span_prune(ctypes.byref(c), _p(q_win), batch, num_q_heads, window,
                                pool_kernel, _p(span), _p(keep_tokens), scale, ctypes.byref(oc),
                                _p(ws), ws.numel(), _stream(stream)), "se_span_prune")


def se_view_sink_recent(kv: PagedKV, batch: int, sink_pages: int, recent_pages: int, view: View,
                        ws, stream=None):
    """The sink + recent pages view of a paged cache."""
    c, vc = kv.c, view.c
    _check(load().se_view_sink_recent(ctypes.byref(c), batch, sink_pages, recent_pages,
                                      ctypes.byref(vc), _p(ws), ws.numel(), _stream(stream)),
           "se_view_sink_recent")


def se_chain_snapshot_bytes(num_seqs: int, num_kv_heads: int, head_dim: int, rows: int,
                            with_score: bool) -> int:
    return load().se_chain_snapshot_bytes(num_seqs, num_kv_heads, head_dim, rows, int(with_score))


def se_chain_save(kv: VarlenKV, seqs, rows: int, snap, ws, stream=None):
    """Copy the retained segments of sequences `seqs` (int32 device) into `snap`."""
    c = kv.c
    _check(load().se_chain_save(ctypes.byref(c), _p(seqs), seqs.numel(), rows, _p(snap),
                                snap.numel(), _p(ws), ws.numel(), _stream(stream)),
           "se_chain_save")


def se_chain_restore(snap, rows: int, seqs, kv: VarlenKV, ws, stream=None):
    """Copy a snapshot's slots into the segments of sequences `seqs` of `kv`."""
    c = kv.c
    _check(load().se_chain_restore(_p(snap), snap.numel(), seqs.numel(), rows, _p(seqs),
                                   ctypes.byref(c), _p(ws), ws.numel(), _stream(stream)),
           "se_chain_restore")


class ChainIndex:
    """The host ChainCacheIndex: logical token prefix -> session id."""

    def __init__(self):
        self._h = load().se_chain_index_create()
        if not self._h:
            raise SparseEngineError("se_chain_index_create failed")

    def close(self):
        if self._h:
            load().se_chain_index_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _tok(tokens):
        import numpy as np
        t = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        return t, t.ctypes.data_as(ctypes.c_void_p), t.size

    def put(self, tokens, sid: int):
        t, ptr, n = self._tok(tokens)
        _check(load().se_chain_index_put(self._h, ptr, n, sid), "se_chain_index_put")

    def match(self, tokens):
        """(id, matched tokens) of the longest stored prefix, (-1, 0) if none."""
        t, ptr, n = self._tok(tokens)
        m = ctypes.c_int64(0)
        sid = load().se_chain_index_match(self._h, ptr, n, ctypes.byref(m))
        if sid < -1:
            _check(int(sid), "se_chain_index_match")
        return int(sid), int(m.value)

    def erase(self, sid: int):
        _check(load().se_chain_index_erase(self._h, sid), "se_chain_index_erase")

    def __len__(self):
        return int(load().se_chain_index_size(self._h))
