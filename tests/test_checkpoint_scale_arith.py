"""The checkpoint scale max / 448 as the activation kernels form it, for every
BF16 maximum from 2^-100 up: q = fl(max c) with c = fl(1/448), then
fl(q + fl(max - 448 q) c), in exact rationals rounded to FP32, equals the
rounded quotient.  (Smaller maxima take the division itself.)"""
from fractions import Fraction

import numpy as np


def fl(v: Fraction) -> Fraction:
    """Nearest FP32 value, ties to even (normal range)."""
    if v == 0:
        return v
    a = abs(v)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    if Fraction(2) ** e > a:
        e -= 1
    step = Fraction(2) ** (e - 23)
    q, r = divmod(a, step)
    if 2 * r > step or (2 * r == step and q % 2):
        q += 1
    return q * step if v > 0 else -q * step


def test_every_bf16_maximum():
    c = fl(Fraction(1, 448))
    # a power of two scales every step exactly: one binade stands for all of
    # them while nothing leaves the normal range (2^-100 / 448 is far above 2^-126)
    for exponent in (-100, -99, 0, 1, 127):
        for m in range(128):
            top = Fraction(128 + m, 128) * Fraction(2) ** exponent
            q = fl(top * c)
            r = fl(top - 448 * q)
            assert fl(q + r * c) == fl(top / 448), (exponent, m)


def test_rounding_helper_is_fp32():
    rng = np.random.default_rng(0)
    for a, b in rng.integers(1, 1 << 24, size=(200, 2)):
        assert float(fl(Fraction(int(a), int(b)))) == float(np.float32(a) / np.float32(b))
