"""Pins of the draft verification oracle."""
from fractions import Fraction

import numpy as np

from oracle import verify as V


def test_every_token_is_distributed_as_the_target():
    """One draft from q, checked against p: over a grid of random numbers that hits each interval by its exact
    length, the first token behind the prefix has p's distribution, whatever q is."""
    p = np.array([0.5, 0.125, 0.25, 0.125, 0.0])
    q = np.array([0.25, 0.25, 0.125, 0.0, 0.375])
    n = 64                                           # all probabilities and ratios are multiples of 1/64
    got = np.zeros(5)
    for d in range(5):
        for i in range(n):
            for j in range(n):
                stay, nxt, keep = V.verify([p, p], [q, q], [9, d], [0, i / n], j / n, 40)
                assert keep == 41 + stay
                got[d if stay else nxt] += q[d] / n / n
    # the residual's grid is exact too: its weights sum to 3/8, thirds of a grid step stay
    assert np.abs(got - p).max() <= 1 / n


def test_draw_is_the_first_sum_that_passes():
    w = [0, 3, 0, 1, 0]
    assert [V.draw(w, u) for u in (0.0, 0.7499, 0.75, 0.99, 1.0, -1.0)] == [1, 1, 3, 3, 3, 1]
    assert V.draw([0, 0], 0.5) is None


def test_whole_numbers_are_the_values():
    x = np.float32([1.0, 0.1, 2.0 ** -149, 1.5 * 2.0 ** -126, 0.0, -0.5, np.nan, 3.0])
    got = [Fraction(w, 2 ** 149) for w in V._whole(x)]
    assert got == [1, Fraction(float(x[1])), Fraction(1, 2 ** 149), Fraction(float(x[3])), 0, 0, 0, 1]


def test_refusals_and_what_is_left():
    p = np.float32([0.5, 0.5, 0.0])
    # looked-up drafts: certain, so u < p decides, and the refused one loses its weight
    assert V.verify([p, p], None, [0, 1], [0, 0.4999], 0.0, 0) == (1, 0, 2)
    assert V.verify([p, p], None, [0, 0], [0, 0.5], 0.0, 0) == (0, 1, 1)
    assert V.verify([p, p], None, [0, 7], [0, 0.0], 0.0, 0) == (0, 0, 1)       # no such token
    # nothing left beside q: drawn from p
    assert V.verify([p, p], [np.float32([1, 1, 1])] * 2, [0, 2], [0, 0.9], 0.9, 5) == (0, 1, 6)
    # the second draft is not looked at behind a refused first
    assert V.verify([p, p, p], None, [0, 2, 0], [0, 0.9, 0.0], 0.0, 0)[0] == 0
    assert V.verify([np.zeros(3)], None, [0], [0], 0.5, 3) == (0, None, 4)
