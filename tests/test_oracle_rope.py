"""Pins of the rotary oracle: closed forms and invariants."""
import math

import numpy as np
import pytest

from oracle import rope as R

FULL = 2 ** 64


def turns_of(f):
    return [round(x / (2 * math.pi) * FULL) for x in f]


def test_a_quarter_turn():
    x = np.arange(1.0, 65.0).reshape(1, 1, 64)
    quarter = [FULL // 4] * 16
    y = R.rotate(x, [1], quarter, layout=R.HALVES)[0, 0]
    assert np.allclose(y[:16], -x[0, 0, 16:32]) and np.allclose(y[16:32], x[0, 0, :16])
    assert np.array_equal(y[32:], x[0, 0, 32:])
    y = R.rotate(x, [1], quarter, layout=R.PAIRS)[0, 0]
    assert np.allclose(y[:32:2], -x[0, 0, 1:32:2]) and np.allclose(y[1:32:2], x[0, 0, :32:2])
    assert np.allclose(R.rotate(x, [4], quarter), x) and np.isnan(R.rotate(x, [-1], quarter)).all()


@pytest.mark.parametrize("layout", [R.HALVES, R.PAIRS])
def test_scores_depend_on_the_distance_alone(layout):
    g = np.random.default_rng(1)
    q, k = g.standard_normal((2, 1, 1, 64))
    t = turns_of(R.frequencies(1e4, 48)[0])
    s = lambda a, b: float(np.sum(R.rotate(q, [a], t, layout=layout) *          # noqa: E731
                                  R.rotate(k, [b], t, layout=layout)))
    for far in (0, 1000, 2 ** 20, 2 ** 30 - 8):
        assert abs(s(far + 7, far) - s(7, 0)) < 1e-9
    assert abs(s(7, 0) - s(9, 0)) > 1e-3


def test_norm():
    g = np.random.default_rng(2)
    x, w = g.standard_normal((3, 2, 64)), g.standard_normal(64)
    y = R.rotate(x, [0, 5, 9], turns_of(R.frequencies(1e4, 64)[0]), weight=np.ones(64), eps=0.0)
    assert np.allclose((y ** 2).mean(-1), 1.0)
    assert np.allclose(R.head_norm(x, w, 0.25), w * x / np.sqrt((x * x).sum(-1, keepdims=True) / 64 + 0.25))
    assert np.allclose(R.rotate(x, [3, 3, 3], turns_of(R.frequencies(1e4, 64)[0]), amp=2.0),
                       2 * R.rotate(x, [3, 3, 3], turns_of(R.frequencies(1e4, 64)[0])))


def test_frequencies():
    f, amp = R.frequencies(1e4, 128)
    assert amp == 1.0 and f[0] == 1.0 and math.isclose(f[32], 1e-2) and len(f) == 64
    assert np.allclose(R.frequencies(1e4, 128, R.LINEAR, 4.0)[0], np.array(f) / 4)
    ntk = R.frequencies(1e4, 128, R.NTK, 4.0)[0]
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 4)       # the slowest pair as if by 1 / factor
    for kind, low, high in ((R.YARN, 1.0, 32.0), (R.BANDS, 1.0, 4.0)):
        y, amp = R.frequencies(5e5, 128, kind, 8.0, 8192.0, low, high)
        plain = np.array(R.frequencies(5e5, 128)[0])
        turns = 8192 * plain / (2 * math.pi)
        ratio = np.array(y) / plain
        assert np.all(np.diff(ratio) <= 1e-12) and ratio[0] == 1.0 and math.isclose(ratio[-1], 1 / 8)
        if kind == R.BANDS:
            assert np.allclose(ratio[turns > high], 1) and np.allclose(ratio[turns < low], 1 / 8)
    assert math.isclose(R.frequencies(1e4, 64, R.YARN, 8.0, 4096.0)[1], 0.1 * math.log(8) + 1)
