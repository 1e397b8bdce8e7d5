"""The oracle's quantiser on rows whose values differ by more than fp64 holds (no
GPU needed)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import history as OH


def tie_row(tiny):
    """A row of bf16 values: `tiny`, values (k + 1/2) steps above 0, and the largest
    that gives the step; and the step."""
    if tiny < 0:
        return np.array([tiny] + [(k + 0.5) * 1.0625 for k in range(8)] + [15.875]), 1.0625
    return np.array([tiny] + [k + 0.5 for k in range(15)] + [15.0]), 1.0


@pytest.mark.parametrize("tiny", [2.0 ** -30, -2.0 ** -30, 2.0 ** -100, -2.0 ** -100, 2.0 ** -133, 0.0])
def test_ties_beside_a_tiny_least_value(tiny):
    """(x - least) / scale just below k + 1/2, just above it, or on it."""
    x, step = tie_row(tiny)
    c, s, lo = OH.quantize_row(x)
    assert s == step and lo == tiny
    assert c.tolist() == [round((Fraction(v) - Fraction(lo)) / Fraction(s)) for v in x]
    halves = c[1:-1].tolist()
    if tiny > 0:
        assert halves == list(range(15))
    elif tiny < 0:
        assert halves == list(range(1, 9))
    else:
        assert halves == [0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14]


def test_the_scale_reaches_the_largest_value():
    for hi, lo in ((15 * 2.0 ** 100, -2.0 ** -100), (15 * 2.0 ** 100, 2.0 ** -100), (15 * 2.0 ** 123, -2.0 ** -120)):
        c, s, _ = OH.quantize_row(np.array([lo, hi]))
        assert Fraction(lo) + 15 * Fraction(s) >= Fraction(hi)
        assert s == hi / 15 * (1 if lo > 0 else 1 + 2.0 ** -7)
