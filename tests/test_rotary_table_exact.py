"""The table of rotary positions holds what the frequencies say, to half of its
unit, so that the last of all positions turns right too (host only)."""
from fractions import Fraction

import numpy as np
import pytest


@pytest.fixture(scope="module")
def bpe():
    import __graft_entry__
    __graft_entry__.build()
    import byte_level_bpe_pretokenize_gb300 as m
    return m


def arctan_of_inverse(n):
    """arctan(1 / n) to 2^-420, by its series."""
    x = Fraction(1, n)
    total, term, k = Fraction(0), x, 1
    while abs(term) > Fraction(1, 2 ** 420):
        total += term / k if k % 4 == 1 else -term / k
        term, k = term * x * x, k + 2
    return total


TWO_PI = 8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))


def off(turn, exact):
    d = (Fraction(int(turn), 2 ** 64) - exact) % 1
    return min(d, 1 - d)


def test_given_frequencies(bpe):
    rng = np.random.default_rng(0)
    f = np.r_[1.0, 0.5, 1e-3, 1e-12, 1e-30, 5e-324, 0.0, -0.0, 6.25, -0.75, -1e-5, -1.0, 100.0, 2 * np.pi, -2 * np.pi,
              np.pi, 1e6, -1e15, 1e22, 2.0 ** 90, rng.normal(0, 1, 300), rng.normal(0, 1, 300) * 10.0 ** rng.integers(-18, 18, 300)]
    for turn, x in zip(bpe.bpe_rotary_table(len(f), frequencies=f), f):
        assert off(turn, Fraction(float(x)) / TWO_PI) <= Fraction(51, 100) / 2 ** 64, x


def test_a_negative_frequency_turns_back(bpe):
    f = np.random.default_rng(1).normal(0, 1, 200)
    a, b = bpe.bpe_rotary_table(200, frequencies=f), bpe.bpe_rotary_table(200, frequencies=-f)
    assert not (a + b).any()


def test_angles_at_the_last_position(bpe):
    """2^-25 of a half turn at position 2^31 - 1, and at -2^31."""
    f = 10_000.0 ** (-np.arange(64) / 64)
    table = bpe.bpe_rotary_table(64, frequencies=f)
    for position in (2 ** 31 - 1, -2 ** 31):
        for turn, x in zip(table, f):
            got = Fraction((int(turn) * position) % 2 ** 64, 2 ** 64)
            d = (got - position * Fraction(float(x)) / TWO_PI) % 1
            assert min(d, 1 - d) <= Fraction(1, 2 ** 33)


def test_frequencies_that_leave_the_doubles(bpe):
    for k in (dict(frequencies=[1.0, 1e300], factor=1e-300), dict(frequencies=[-1e300, 0.0], factor=1e-200)):
        with pytest.raises(bpe.BpeError) as e:
            bpe.bpe_rotary_table(2, **k)
        assert e.value.code == 1 and "finite" in str(e.value)
    assert bpe.bpe_rotary_table(2, frequencies=[1.7e308, -1.7e308]).shape == (2,)
