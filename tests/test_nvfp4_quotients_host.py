"""The 4-bit quantiser divides by a corrected reciprocal (csrc/nvfp4_quant.cuh):
r = 1 / den, q = x r, then q + r (x - q den), each rounded to binary32.  In
rational arithmetic, for every 8-bit significand x and every divisor for which
x / den comes within two units in the last place of a border between two E2M1
codes: the result is the division's.  Elsewhere one unit more or less leaves
the code as it is, which a sample of other quotients bounds."""
import math
import random
from fractions import Fraction as F

import pytest

BORDERS = [F(1, 4), F(3, 4), F(5, 4), F(7, 4), F(5, 2), F(7, 2), F(5)]
ONE = 2 ** 23                     # significands of a divisor in [1, 2): ONE .. 2 ONE - 1, all ones excluded


def exponent(v):
    e = v.numerator.bit_length() - v.denominator.bit_length()
    return e if F(2) ** e <= v else e - 1


def rn(v):
    """Binary32, nearest even (normal range)."""
    if v == 0:
        return F(0)
    unit = F(2) ** (exponent(abs(v)) - 23)
    return round(v / unit) * unit          # (round of a Fraction: half to even)


def both(x, den):
    r = rn(1 / den)
    q = rn(x * r)
    return rn(q + r * rn(x - q * den)), rn(x / den), q


@pytest.mark.parametrize("border", BORDERS)
def test_quotients_at_a_border(border):
    checked = 0
    for m in range(128, 256):
        x = F(m)
        e = exponent(x / border)
        x = x / F(2) ** e                                  # x / border in [1, 2)
        near = math.floor(x / border * ONE)
        for k in range(max(ONE, near - 5), min(2 * ONE - 2, near + 6) + 1):
            got, want, _ = both(x, F(k, ONE))
            assert got == want, (m, k)
            checked += 1
    assert checked > 128 * 5
    # five steps of the divisor are past two units of the quotient
    unit = F(2) ** (exponent(border) - 23)
    for c in (F(ONE + 6, ONE), F(3, 2), F(2 * ONE - 8, ONE)):
        assert abs(border * c / (c + F(6, ONE)) - border) > 2 * unit


def test_other_quotients_are_within_a_unit():
    rng = random.Random(1)
    for _ in range(20000):
        x, den = F(rng.randrange(128, 256)), F(rng.randrange(ONE, 2 * ONE - 1), ONE)
        got, want, q = both(x, den)
        unit = F(2) ** (exponent(want) - 23)
        assert abs(q - x / den) <= F(3, 2) * unit and abs(got - want) <= unit
