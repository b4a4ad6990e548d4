"""The cache write's quotient: with y = RN(1 / scale), q = RN(x y) and r = RN(x - q scale), RN(q + r y) is
RN(x / scale) in float32 for every bf16 element x of a row whose largest element is bf16 too. While nothing leaves
the normal range, powers of two do not matter: 128 significands of the row's largest element (scale = RN(it / 448))
and 128 of x are all there are."""
from fractions import Fraction

import numpy as np


def rn(v: Fraction) -> Fraction:
    """v rounded to 24 significant bits, ties to even."""
    if v == 0:
        return v
    a = abs(v)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    if Fraction(2) ** e > a:
        e -= 1
    elif Fraction(2) ** (e + 1) <= a:
        e += 1
    unit = Fraction(2) ** (e - 23)
    return (1 if v > 0 else -1) * round(a / unit) * unit  # (round() of a Fraction is to even)


def test_rounding_is_float32s():
    rng = np.random.default_rng(0)
    for a, b in rng.integers(1, 1 << 24, (500, 2)):
        assert Fraction(float(np.float32(int(a)) / np.float32(int(b)))) == rn(Fraction(int(a), int(b)))


def test_every_pair_of_significands():
    for top in range(128, 256):
        scale = rn(Fraction(top, 448))
        y = rn(1 / scale)
        for x in range(128, 256):
            q = rn(x * y)
            r = rn(x - q * scale)
            assert rn(q + r * y) == rn(x / scale), (top, x)
