"""The quotients that FP8_BLOCK blocks are rounded from: z = x inv, r = x - z s, z + r inv, with
inv = 1 / s, every operation rounded to fp32 once (a fused one as a whole), against x / s rounded
to fp32 once.  A scale is m / 448 and x is bf16, both of 8 significant bits; powers of two move
nothing, so 128 x 128 significands are all that there are."""
from fractions import Fraction

import pytest


def _fp32(x):
    """The nearest number of 24 significant bits, ties to even."""
    if x == 0:
        return Fraction(0)
    e = abs(x.numerator).bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > abs(x):
        e -= 1
    unit = Fraction(2) ** (e - 23)
    return round(x / unit) * unit


@pytest.mark.parametrize("part", range(4))
def test_quotients_of_every_pair_of_significands(part):
    for m in range(128 + 32 * part, 160 + 32 * part):
        s = _fp32(Fraction(m, 448))
        inv = _fp32(1 / s)
        for n in range(128, 256):
            x = Fraction(n) if n <= m else Fraction(n, 2)
            z = _fp32(x * inv)
            assert _fp32(z + _fp32(x - z * s) * inv) == _fp32(x / s), (n, m)
