"""Rotary positions with norms of queries and keys per head (oracle).

Pairs (a, b) of a head's first rot channels, (i, i + rot / 2) or (2i, 2i + 1), turn by the angle
2 pi * (pos * turns[i] mod 2^64) / 2^64: (amp * (a cos - b sin), amp * (b cos + a sin)).  Before
that, with a weight, x becomes x * w / sqrt(mean(x^2) + eps) over the head.  float64; the angle's
fraction of a turn in whole numbers.
"""
import math

import numpy as np

HALVES, PAIRS = 0, 1
PLAIN, LINEAR, NTK, YARN, BANDS = range(5)


def frequencies(base, rot, kind=PLAIN, factor=1.0, length=0.0, low=1.0, high=32.0):
    """(radians a position of each pair, amplitude)."""
    if kind == NTK:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if kind == LINEAR:
        return [x / factor for x in f], 1.0
    if kind == YARN:
        def index(turns):                    # of the pair that turns so often over the length
            return rot * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(index(high))), min(rot - 1, math.ceil(index(low)))
        slow = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        return ([x * (1 - s) + x / factor * s for x, s in zip(f, slow)],
                0.1 * math.log(factor) + 1)
    if kind == BANDS:
        fast = [min(1.0, max(0.0, (length * x / (2 * math.pi) - low) / (high - low))) for x in f]
        return [x * s + x / factor * (1 - s) for x, s in zip(f, fast)], 1.0
    return f, 1.0


def head_norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x * np.asarray(weight, dtype=np.float64) / np.sqrt(
        (x ** 2).mean(-1, keepdims=True) + eps)


def pairs_of(rot, layout):
    """The two channels of each pair."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == HALVES else (2 * i, 2 * i + 1)


def rotate(x, pos, turns, amp=1.0, layout=HALVES, weight=None, eps=1e-6):
    """x [rows][heads][D], pos [rows] -> the rows with pos >= 0 normed and turned, others NaN."""
    y = head_norm(x, weight, eps).copy()
    a, b = pairs_of(2 * len(turns), layout)
    for t, p in enumerate(pos):
        if p < 0:
            y[t] = np.nan
            continue
        angle = np.array([2 * math.pi * (int(p) * int(w) % 2 ** 64) / 2 ** 64 for w in turns])
        u, v = y[t][:, a].copy(), y[t][:, b].copy()
        y[t][:, a] = amp * (u * np.cos(angle) - v * np.sin(angle))
        y[t][:, b] = amp * (v * np.cos(angle) + u * np.sin(angle))
    return y


def rounding_bound(x, want, rot, amp, layout, weight, eps):
    """Largest difference of a bf16 result computed in fp32 from `want`: its rounding (half a step, 2^-8
    of the value) and the fp32 terms, relative to amp (|a| + |b|) of the pair: angle 9.4e-8 (an
    fp32 fraction of a half turn, times pi), cosine and amplitude 2.4e-7, the norm's sum of 128 squares in a
    tree (at most 17 + 5 roundings, half of them under the root) 6.6e-7, reciprocal root 2.4e-7, products 3e-7;
    together below 2e-6."""
    y = np.abs(head_norm(x, weight, eps))
    reach = y.copy()
    a, b = pairs_of(rot, layout)
    reach[..., a] = reach[..., b] = abs(amp) * (y[..., a] + y[..., b])
    return 2.0 ** -8 * np.abs(want) + 2e-6 * (1 + 2.0 ** -8) * reach
