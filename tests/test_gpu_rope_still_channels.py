"""GPU tests of the channels that a rotation leaves alone: they keep their values, whatever lies beside them."""
import math

import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from tests.test_gpu_chunk import both_pools, i32, plan_both
from tests.test_gpu_rope import bf16, make, marked, small_ws

pytestmark = pytest.mark.gpu
SHAPES = [(128, 0), (128, 16), (128, 96), (64, 0), (64, 48)]       # channels of a head, rotated ones


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


def bits(x):
    return x.contiguous().view(torch.int16)


def same(a, b):
    """The same bits, NaN for NaN."""
    return bool(((bits(a) == bits(b)) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("layout", [se.SE_ROPE_HALVES, se.SE_ROPE_PAIRS])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_without_a_norm_they_are_what_they_were(dim, rot, layout):
    """Infinities, NaN and negative zeros in one of them: the others, and the rotated ones, do not see it.
    Rows of one pass (two heads) and of several."""
    g = np.random.default_rng([41, dim, rot, layout])
    rope = make(g, rot, dim, layout, (0, 0), amp=1.25)
    pos = [0, 5, 70000, 2 ** 31 - 1]
    for heads in (2, 37):
        x = bf16(g, 4, heads, dim)
        clean = marked(4, heads, dim)
        se.se_qk_rope(rope, i32(pos), x, None, clean, None, small_ws())
        assert same(clean[..., rot:], x[..., rot:])
        for bad in (math.inf, -math.inf, math.nan, -0.0):
            for c in {rot, rot + 1, rot + 8, (rot + dim) // 2, dim - 1}:
                y, out = x.clone(), marked(4, heads, dim)
                y[:, 1, c] = bad
                se.se_qk_rope(rope, i32(pos), None, y, None, out, small_ws())
                assert same(out[..., rot:], y[..., rot:]), (bad, c)
                assert same(out[..., :rot], clean[..., :rot]), (bad, c)


@pytest.mark.parametrize("layout", [se.SE_ROPE_HALVES, se.SE_ROPE_PAIRS])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_with_a_norm_as_its_formula(dim, rot, layout):
    """x w / sqrt(mean x^2 + eps) of a row with an infinity: 0 for the finite ones, NaN for itself."""
    g = np.random.default_rng([42, dim, rot, layout])
    rope = make(g, rot, dim, layout, (1, 0))
    x = bf16(g, 3, 4, dim)
    clean = marked(3, 4, dim)
    se.se_qk_rope(rope, i32([1, 2, 3]), x, None, clean, None, small_ws())
    for c in {rot, rot + 8, dim - 1}:
        for bad in (math.inf, -math.inf, math.nan):
            y, out = x.clone(), marked(3, 4, dim)
            y[1, 2, c] = bad
            se.se_qk_rope(rope, i32([1, 2, 3]), y, None, out, None, small_ws())
            head = out[1, 2].clone()
            if math.isnan(bad):
                assert head.isnan().all()
            else:
                assert head[c].isnan()
                head[c] = 0
                assert (head == 0).all(), (c, bad)
            out[1, 2] = clean[1, 2]
            assert same(out, clean)


@pytest.mark.parametrize("layout", [se.SE_ROPE_HALVES, se.SE_ROPE_PAIRS])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_appended_keys_and_their_summaries(dim, rot, layout):
    g = np.random.default_rng([43, dim, rot, layout])
    o, p = both_pools(8, 2, 4)
    rope = make(g, rot, dim, layout, (0, 0))
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")              # noqa: E731
    kv = se.PagedKV(z(8, 3, 16, dim), z(8, 3, 16, dim), z(2, 4, 3, 2, dim), p.block_table, p.ctx_len)
    chunk = plan_both(o, p, [20, 3], 23, se.workspace(se.se_page_pool_workspace(2)))
    x = bf16(g, 23, 8, dim)
    k = x[:, 2:5]
    k[4, 1, rot] = math.inf
    k[7, 1, dim - 1] = math.nan
    k[17, 2, rot + 8] = -math.inf
    k[20:, 0, (rot + dim) // 2] = -0.0
    qo = marked(23, 2, dim)
    se.se_rope_append_chunk(kv, rope, x[:, :2], k, x[:, 5:], qo, chunk, 2, small_ws())
    assert same(qo[..., rot:], x[:, :2, rot:])
    slots = chunk.slot.tolist()
    rows = torch.stack([kv.k[s // 16, :, s % 16] for s in slots])
    assert same(rows[..., rot:], k[..., rot:]) and not rows[..., :rot].isnan().any()
    for b, page, first, last in ((0, 0, 0, 16), (0, 1, 16, 20), (1, 0, 20, 23)):
        seen = rows[first:last].float()
        low, high = seen.nan_to_num(math.inf, math.inf, -math.inf), seen.nan_to_num(-math.inf, math.inf, -math.inf)
        assert kv.meta[b, page, :, 0].float().equal(low.amin(0))
        assert kv.meta[b, page, :, 1].float().equal(high.amax(0))
