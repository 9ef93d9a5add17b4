"""se_chunk_attn on numbers at the edges of what it takes: the largest logits, and rows of q
behind the last sequence that are no numbers."""
import numpy as np
import pytest
import torch

from kv_cache_decode_quest_gb300 import binding as se
from tests.test_gpu_chunk import Attn, Cache, bf16, f64, held, normal, plan_both

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    return lib


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 29])
def test_largest_logits(top, f32):
    """Logits of +-top and 0, all exact in fp32: the keys at a row's largest logit share it, all
    others get nothing.  The reference that is taken off is a rounded product of size
    t = top log2 e, so every weight at the top is one and the same number 2^e, |e| <= 2^-24 t
    (at most 2^32 for 2^29), which divides out: P is a power of two up to ex2's relative
    2^-22 and its rounding (2^-8, or 2^-16 in two terms), the sums of n equal terms round
    by 2^-23 each at most, and 2^-8 or 2^-24 of the result its own type."""
    g = np.random.default_rng([71])
    n, D = 300, 64
    c = Cache(g, 1, 1, D, 20, 20)
    k = np.zeros((n, 1, D))
    level = g.integers(-1, 2, n)
    level[:140] = np.minimum(level[:140], 0)               # the top comes after the first tile
    k[:, 0, 0] = level * 2.0 ** 10
    v = normal(g, n, 1, D)
    chunk = plan_both(c.o, c.pool, [n], n, c.ws_pool)
    se.se_kv_append_chunk(c.kv, bf16(k), bf16(v), chunk, 1, c.ws)
    a = Attn(c, 2, f32, scale=top * 2.0 ** -20)
    a.run(chunk)
    q = np.zeros((n, 2, D))
    q[..., 0] = 2.0 ** 10
    a.qt = bf16(q)
    a.call(chunk)
    assert se.status_word(a.ws) == 0
    out, lse = f64(a.out), f64(a.lse)
    for i in range(n):
        at = np.flatnonzero(level[:i + 1] == level[:i + 1].max())
        want, size = v[at, 0].mean(0), np.abs(v[at, 0]).mean(0)
        tol = size * ((2.0 ** -16 if f32 else 2.0 ** -8) + 2.0 ** -21 + len(at) * 2.0 ** -22) + \
            np.abs(want) * (2.0 ** -24 if f32 else 2.0 ** -8)
        assert np.all(np.abs(out[i] - want) <= tol), i
        z = level[:i + 1].max() * top + np.log(len(at))
        assert np.all(np.abs(lse[i] - z) <= 2.0 ** -22 * (np.abs(z) + 2)), i


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3e38])
def test_rows_behind_the_last_sequence_may_hold_anything(fill):
    """They share tiles of rows with the last sequence, whose results keep their bits."""
    g = np.random.default_rng([72])
    for D, G, ctx, new in ((64, 2, [300, 500], [5, 37]), (128, 8, [100, 2000], [40, 3])):
        c = held(g, 2, 2, D, ctx, new)
        chunk = c.add(new, pad=70)
        a = Attn(c, G)
        a.run(chunk)
        a.check(chunk, rows=20)
        out, lse, rows = a.out.clone(), a.lse.clone(), sum(new)
        a.qt[rows:] = fill
        a.out.fill_(7)
        a.lse.fill_(7)
        a.call(chunk)
        assert se.status_word(a.ws) == 0
        assert torch.equal(a.out, out) and torch.equal(a.lse, lse)
