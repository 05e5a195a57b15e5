"""The arithmetic by which mt_token_probs takes an exponential's argument to
twice fp32 (Exp2::of and log2_scale), in exactly rounded fp32 steps against
rationals."""
from fractions import Fraction
import math

import numpy as np


def rounded(x):
    """The nearest float of a rational, the even one of two (no subnormals here)."""
    if x == 0:
        return Fraction(0)
    s, x = (-1 if x < 0 else 1), abs(x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    step = Fraction(2) ** (e - 23)
    n = x / step
    low = n.numerator // n.denominator
    part = n - low
    if part > Fraction(1, 2) or (part == Fraction(1, 2) and low % 2):
        low += 1
    return s * low * step


def fma(a, b, c):
    return rounded(a * b + c)


def scale(t, off):
    """hi, lo of log2(e) / t; off: the reciprocal's error in steps of 2^-24."""
    l_hi, l_lo = Fraction(float(np.float32(1.44269502))), Fraction(float(np.float32(1.92596303e-8)))
    r = rounded(1 / t * (1 + off * Fraction(1, 2 ** 24)))
    hi = rounded(l_hi * r)
    return hi, rounded(rounded(fma(-hi, t, l_hi) + l_lo) * r)


def argument(d, hi, lo):
    """y and rest, of which y + rest stands for 40 + d (hi + lo)."""
    y = rounded(fma(d, hi, 384) - 344)
    return y, fma(d, lo, fma(d, hi, rounded(40 - y)))


# log2(e) to 100 bits: e from its series, the logarithm bit by bit
def log2e(bits=100):
    e = sum(Fraction(1, math.factorial(n)) for n in range(60))
    x, out = e / 2, Fraction(1)
    for k in range(1, bits):
        x = x * x
        x = Fraction(x.numerator * 2 ** 300 // x.denominator, 2 ** 300)
        if x >= 2:
            out += Fraction(1, 2 ** k)
            x /= 2
    return out


def test_the_argument_is_exact_to_twice_fp32():
    L = log2e()
    assert abs(float(L) - math.log2(math.e)) < 1e-15
    rng = np.random.default_rng(1)
    for t in (1.0, 0.7, 0.01, 3.0, 1e-6, 1e6):
        t = Fraction(float(np.float32(t)))
        for off in (-1, 0, 1):
            hi, lo = scale(t, off)
            for z in np.concatenate([-rng.random(150) * 199, -np.exp(-12 * rng.random(50)), [-40.0, -39.999, -24.0, -56.0, -128.0, -199.9]]):
                d = Fraction(float(np.float32(z / float(hi))))
                y, rest = argument(d, hi, lo)
                want = 40 + d * L / t
                # 2^-40 of the product and of 1; the rest: half a step of 2^-15, and d lo, lo being hi's
                # rounding (2^-24) and the reciprocal's error (2^-23): 2^-16 + 200 * 1.5 * 2^-23 < 2^-14
                assert abs(y + rest - want) <= Fraction(1, 2 ** 40) * (1 + abs(d * hi)), (float(t), float(d))
                assert abs(rest) < Fraction(1, 2 ** 14)
