"""The divisions of the 4-bit cache's quantiser, emulated with exact fractions (no GPU needed).

quant8 (kv4_layout.cuh) divides by a scale of 8 significant bits: r = one Newton step from the
hardware's approximate reciprocal (off by at most one unit in the last place), q = RN(a r),
then RN(q + (a - q b) r), each step one fused multiply-add. By Markstein's theorem the last is
the correctly rounded quotient if r is the correctly rounded reciprocal."""

from __future__ import annotations

from fractions import Fraction

import pytest


def rn(x: Fraction) -> Fraction:
    """x rounded to 24 significant bits, ties to even (no limit on the exponent)."""
    if x == 0:
        return x
    s, x = (-1, -x) if x < 0 else (1, x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    unit = Fraction(2) ** (e - 23)
    return s * round(x / unit) * unit  # Python rounds halves to even


def fma(a, b, c):
    return rn(a * b + c)


SCALES = [Fraction(m, 128) for m in range(128, 256)]


def near(x: Fraction):
    """The values within two units in the last place of a rounded x in (1/2, 1]."""
    return [x + j * Fraction(1, 2 ** 24) for j in range(-2, 3)]


def test_rn_itself():
    import numpy as np

    rng = np.random.default_rng(0)
    for a, b in zip(rng.integers(1, 2 ** 60, 500), rng.integers(1, 2 ** 23, 500)):
        assert rn(Fraction(int(a))) == Fraction(float(np.float32(int(a))))
        assert rn(Fraction(1, int(b))) == Fraction(float(np.float32(1) / np.float32(int(b))))


def test_reciprocal_of_every_scale_is_correctly_rounded():
    """From any start within two units in the last place (the hardware's is within one)."""
    for b in SCALES:
        want = rn(1 / b)
        for y in near(want):
            assert fma(fma(-b, y, Fraction(1)), y, y) == want, b


def quotient(a, b, r):
    q = rn(a * r)
    return fma(fma(-q, b, a), r, q)


@pytest.mark.parametrize("part", range(8))
def test_quotients_are_correctly_rounded(part):
    """Every scale against numerators of up to 10 significant bits (differences of bf16 values
    of one size have 9), and the multiples of half a step, where codes change."""
    for b in SCALES[part::8]:
        r = rn(1 / b)
        for a in [Fraction(n, 512) for n in range(512, 1024)] + [b * n / 2 for n in range(1, 31)]:
            assert quotient(a, b, r) == rn(a / b)


def test_ranges_by_fifteen_are_correctly_rounded():
    b, r = Fraction(15), rn(Fraction(1, 15))
    for n in range(2 ** 12, 2 ** 13):
        a = Fraction(n, 2 ** 12)
        assert quotient(a, b, r) == rn(a / b)
