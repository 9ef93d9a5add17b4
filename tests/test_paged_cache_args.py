"""The binding's look at a paged cache: tables, pages or summaries that a call would write past, or read as
something else, are refused on the host."""
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding
from tests.test_chunk_args import NoStream, cache_of, chunk_of, lib  # noqa: F401

pytestmark = pytest.mark.usefixtures("lib")
WS = torch.zeros(1 << 12, dtype=torch.uint8)


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def refused(match):
    return pytest.raises(binding.SparseEngineError, match=match)


def rope_append(kv, batch=2):
    binding.se_rope_append_chunk(kv, binding.Rope(None, 0), None, z(8, 2, 64), z(8, 2, 64), None,
                                 chunk_of(batch=batch), batch, WS, stream=NoStream)


def append(kv, batch=2):
    binding.se_kv_append_chunk(kv, z(8, 2, 64), z(8, 2, 64), chunk_of(batch=batch), batch, WS[:8],
                               stream=NoStream)


def carry(kv, batch=2):
    binding.se_pages_carry(kv, binding.Carry.empty(batch, "cpu"), batch, WS, stream=NoStream)


def attn(kv, batch=2):
    q = z(8, 4, 64)
    binding.se_chunk_attn(kv, q, chunk_of(batch=batch), batch, 4, 1.0, q.clone(), None, WS[:8], stream=NoStream)


CALLS = [(rope_append, "current CUDA device"), (append, "workspace"), (carry, "current CUDA device"),
         (attn, "workspace")]                       # and what each says of a cache that is right


@pytest.mark.parametrize("call,passed", CALLS)
def test_pages_and_tables(call, passed):
    for good in (cache_of(), cache_of(meta=z(2, 4, 2, 2, 64)), cache_of(batch=5)):
        with refused(passed):
            call(good)
    for field, bad, says in (("v", z(3, 2, 16, 64), "one shape"), ("v", z(4, 1, 16, 64), "one shape"),
                             ("v", z(4, 16, 2, 64).transpose(1, 2), "one shape"),
                             ("v", z(4, 2, 16, 64, dtype=torch.float16), "bfloat16"),
                             ("block_table", z(2, 4, dtype=torch.int64), "block_table.*int32"),
                             ("block_table", z(2, 8, dtype=torch.int32)[:, ::2], "block_table.*int32"),
                             ("block_table", z(2, 4, 1, dtype=torch.int32), "block_table.*int32"),
                             ("ctx_len", z(2, dtype=torch.int64), "ctx_len.*int32"),
                             ("ctx_len", z(4, dtype=torch.int32)[::2], "ctx_len.*int32"),
                             ("ctx_len", z(1, dtype=torch.int32), "too short for 2")):
        kv = cache_of()
        with refused(passed):
            call(kv)
        setattr(kv, field, bad)                     # (also when it is put there later)
        with refused(says):
            call(kv)


@pytest.mark.parametrize("call,passed", CALLS[:3])
def test_summaries_that_are_written(call, passed):
    for bad in (z(1, 4, 2, 2, 64), z(2, 3, 2, 2, 64), z(2, 4, 1, 2, 64), z(2, 4, 2, 2, 128), z(2, 4, 2, 64),
                z(1), z(2, 4, 2, 64, 2).transpose(3, 4), z(4, 4, 2, 2, 64)[::2]):
        with refused("PagedKV.meta"):
            call(cache_of(meta=bad))
    with refused(passed):                           # more sequences than the call names
        call(cache_of(batch=3, meta=z(2, 4, 2, 2, 64)))
    with refused("PagedKV.meta"):
        call(cache_of(batch=3, meta=z(2, 4, 2, 2, 64)), batch=3)


def test_summaries_that_nobody_touches():
    with refused("workspace"):
        attn(cache_of(meta=z(1)))
