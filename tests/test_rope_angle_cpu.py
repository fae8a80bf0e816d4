"""The bound that the header gives for a rotary angle, from the method's own arithmetic in whole
numbers: freq / 2 pi in units of 2^-64 turns, rounded down, times the position modulo 2^64,
rounded to 32 bits."""
import math
import random
from fractions import Fraction

import pytest


def two_pi():
    one = 1 << 300

    def arctan_inverse(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (term if k % 2 == 0 else -term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total

    return Fraction(2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)


TWO_PI = two_pi()
A = math.floor(2 ** 66 / TWO_PI)  # 1 / 2 pi in units of 2^-66


def error(freq, t):
    """How far the angle is off, in turns."""
    unit = math.floor(abs(Fraction(freq)) * A / 4)  # in units of 2^-64
    turns = (unit if freq >= 0 else -unit) * t % 2 ** 64
    kept = Fraction((turns + 2 ** 31) // 2 ** 32, 2 ** 32)
    off = kept - Fraction(freq) * t / TWO_PI
    return abs(off - round(off))


def bound(freq, t):
    return abs(t) * (Fraction(1, 2 ** 64) + abs(Fraction(freq)) / 2 ** 66) + Fraction(1, 2 ** 33)


@pytest.mark.parametrize("seed", range(20))
def test_bound(seed):
    rng = random.Random(seed)
    for _ in range(200):
        freq = math.ldexp(rng.uniform(1, 2) * rng.choice([-1, 1]), rng.randint(-70, 53))
        t = rng.choice([rng.randint(-2 ** 31, 2 ** 31 - 1), rng.randint(0, 1 << 17), 2 ** 31 - 1, -2 ** 31])
        assert error(freq, t) <= bound(freq, t)
        if abs(t * Fraction(freq)) <= 2 ** 32:
            assert error(freq, t) * TWO_PI < Fraction(1, 2 ** 29)


def test_the_bound_is_near():
    """Frequencies below 2^-8 lose, at far positions, what the unit of 2^-64 leaves."""
    rng = random.Random(1)
    t = 2 ** 31 - 1
    assert max(float(error(f, t) / bound(f, t)) for f in
               (math.ldexp(rng.uniform(1, 2), -9) for _ in range(300))) > 0.5
