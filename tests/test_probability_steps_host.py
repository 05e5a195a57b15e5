"""The arithmetic by which mt_tree_verify takes probabilities in steps of 2^-56
(fp32 sums with 12, 1.5 2^-17 and 1.5 2^-33), against rationals."""
from fractions import Fraction

import numpy as np


def steps(p):
    """The kernel's integer for p in [-1, 1], in fp32 operations."""
    f, total, left = np.float32, 0, np.float32(p)
    for magic, shift in ((f(12), 36), (f(1.5 * 2 ** -17), 16), (f(1.5 * 2 ** -33), 0)):
        y = f(left + magic)
        total += (int(y.view(np.uint32)) - int(magic.view(np.uint32))) << shift
        left = f(left - f(y - magic))
    return total


def nearest(x):
    """The nearest integer, the even one of two."""
    low = x.numerator // x.denominator
    part = x - low
    return low if part < Fraction(1, 2) or (part == Fraction(1, 2) and low % 2 == 0) else low + 1


def test_steps_are_the_nearest_integers():
    rng = np.random.default_rng(1)
    p = np.concatenate([rng.random(3000), np.exp(-60 * rng.random(5000)), 2.0 ** -np.arange(0, 70), 1.5 * 2.0 ** -np.arange(1, 70),
                        [0, 1 - 2 ** -24, 2 ** -21 + 2 ** -44, 2.5 * 2 ** -56, 2 ** -149]]).astype(np.float32)
    assert [m.view(np.uint32) for m in (np.float32(12), np.float32(1.5 * 2 ** -17), np.float32(1.5 * 2 ** -33))] == [0x41400000, 0x37400000, 0x2F400000]
    for x in p:
        want = nearest(Fraction(float(x)) * 2 ** 56)
        assert steps(x) == want and steps(-x) == -want, x
        assert x < 2 ** -33 or want == Fraction(float(x)) * 2 ** 56  # exact where a float's own step is larger
