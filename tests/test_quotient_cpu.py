"""The cache's quotient: q = RN(x y), RN(q + RN(x - q s) y) with y = RN(1 / s) is the correctly rounded x / s for
every mantissa of a bf16 x and every scale s = RN(amax / 448) of a bf16 amax (exponents only shift all of it)."""

from fractions import Fraction

import numpy as np


def rn32(x: Fraction) -> Fraction:
    """Nearest fp32 to a positive rational, ties to even (no under- or overflow)."""
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    assert Fraction(2) ** e <= x < Fraction(2) ** (e + 1)
    step = Fraction(2) ** (e - 23)
    return round(x / step) * step  # Fraction's round is to even


def signed(x: Fraction) -> Fraction:
    return Fraction(0) if x == 0 else rn32(x) if x > 0 else -rn32(-x)


def test_every_mantissa():
    for a in range(128, 256):
        s = rn32(Fraction(a, 448))
        y = rn32(1 / s)
        for m in range(128, 256):
            x = Fraction(m)
            q = rn32(x * y)
            r = signed(x - q * s)
            assert signed(q + r * y) == rn32(x / s), (a, m)


def test_rounding_helper_matches_fp32():
    rng = np.random.default_rng(1)
    for _ in range(500):
        n, d = int(rng.integers(1, 1 << 24)), int(rng.integers(1, 1 << 24))
        assert float(rn32(Fraction(n, d))) == float(np.float32(n) / np.float32(d))
