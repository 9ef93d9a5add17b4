"""Drafted tokens against the target's probabilities (oracle), in exact arithmetic.

Draft d behind row t stays while u q[t][d] < p[t][d]; behind the first refused one (row r) the next
token is drawn from max(0, p[r] - q[r]), behind the last row from p, as the first token whose running sum passes
u times the whole.  Without q a draft counts as certain: q is 1 for it and 0 elsewhere.
"""
from fractions import Fraction

import numpy as np

BELOW_ONE = 1 - 2.0 ** -24


def _whole(x):
    """A row of fp32 values as integers in units of 2^-149; NaN and negative ones 0, at most 1."""
    x = np.asarray(x, dtype=np.float64)
    x = np.minimum(np.where(x > 0, x, 0.0), 1.0)
    m, e = np.frexp(x)
    return [int(a * 2 ** 24) << (int(b) - 24 + 149) if b >= 24 - 149 else
            int(a * 2 ** 24) >> (24 - 149 - int(b)) for a, b in zip(m, e)]


def draw(weights, u):
    """The first index whose running sum passes u * sum; None without any weight."""
    total = sum(weights)
    if total == 0:
        return None
    want = Fraction(float(min(max(u, 0.0), BELOW_ONE))) * total
    run = 0
    for v, w in enumerate(weights):
        run += w
        if run > want:
            return v


def verify(p, q, tokens, accept_u, sample_u, first):
    """One sequence's rows p [n][V], q the same or None, tokens [n], accept_u [n]; `first` the position of
    its first row.  Returns (accepted, next token, length to keep); the token is None without any weight."""
    n, V = np.shape(p)
    stay = 0
    while stay < n - 1:
        d = int(tokens[stay + 1])
        u = Fraction(float(min(max(accept_u[stay + 1], 0.0), BELOW_ONE)))
        if not 0 <= d < V or np.isnan(p[stay][d]):
            break
        chance = Fraction(1) if q is None else Fraction(float(q[stay][d]))
        if not u * chance < Fraction(float(p[stay][d])):
            break
        stay += 1
    w = whole = _whole(p[stay])
    if stay < n - 1:
        if q is not None:
            w = [max(0, a - b) for a, b in zip(whole, _whole(q[stay]))]
        else:
            w = list(whole)
            if 0 <= int(tokens[stay + 1]) < V:
                w[int(tokens[stay + 1])] = 0
        if sum(w) == 0:
            w = whole
    return stay, draw(w, sample_u), first + 1 + stay
