"""Frequencies as whole 2^-64 turns against f / 2 pi in whole numbers, on the CPU."""
import math
from fractions import Fraction

import pytest

BITS = 1400  # of 1 / 2 pi behind the point


@pytest.fixture(scope="module")
def va():
    from packed_variable_length_varlen_gb300 import build
    build.build()
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


def _inverse_two_pi():
    """1 / 2 pi as a fraction, by Machin's formula: pi / 4 = 4 atan(1 / 5) - atan(1 / 239)."""
    one = 1 << (BITS + 64)

    def atan_of_inverse(x):
        total, term, k, sign = 0, one // x, 1, 1
        while term:
            total += sign * (term // k)
            term //= x * x
            k, sign = k + 2, -sign
        return total

    return Fraction(one, 8 * (4 * atan_of_inverse(5) - atan_of_inverse(239)))


INVERSE = _inverse_two_pi()


def _off(f, t):
    """How far t is from f / 2 pi * 2^64 modulo 2^64."""
    d = (Fraction(f) * INVERSE * 2 ** 64 - t) % 2 ** 64
    return float(min(d, 2 ** 64 - d))


def test_the_inverse_itself():
    assert abs(float(INVERSE) - 1 / (2 * math.pi)) < 1e-16


def _frequencies():
    f = [500000.0 ** (-i / 20000) for i in range(0, 20000, 7)] + [10000.0 ** (-2 * i / 128) for i in range(64)]
    f += [1.0, 2 * math.pi, math.pi, 100.0, 12345.678, 1048575.9, 2.0 ** -40, 2.0 ** -61, 1e-30, 5e-324, 0.0]
    f += [math.nextafter(2 * math.pi, 0), math.nextafter(2 * math.pi, 10), 2 * math.pi * 1000]
    return f + [-x for x in f]


def test_turns_are_rounded_once(va):
    """Half a unit, and for |f| < 2^20 no more than 2^-20 of one from the sums on the way (f / 2 pi < 2^18 in two doubles is
    good to 2^-104 of it, 2^-22 units; what is left of 2^-64 turns is added up below 2^30 units, in steps of 2^-23)."""
    f = _frequencies()
    st, turns = va.varlen_attn_rotary_turns(f)
    assert st == 0 and all(0 <= t < 2 ** 64 for t in turns)
    worst = max((_off(x, t), x) for x, t in zip(f, turns))
    assert worst[0] <= 0.5 + 2.0 ** -20, worst


def test_turns_change_their_sign_with_the_frequency(va):
    f = _frequencies()
    half = len(f) // 2
    turns = va.varlen_attn_rotary_turns(f)[1]
    assert [(-t) % 2 ** 64 for t in turns[:half]] == turns[half:]


def test_angles_of_far_positions(va):
    """What the header says of any int32 position: from turns within half a unit (and a little), 2^31 times that."""
    f = [500000.0 ** (-i / 64) for i in range(64)]
    f += [-x for x in f]
    turns = va.varlen_attn_rotary_turns(f)[1]
    for p in (2 ** 31 - 1, -2 ** 31, 2 ** 24 + 3):
        for x, t in zip(f, turns):
            d = (Fraction(x) * INVERSE * p - Fraction(p * t, 2 ** 64)) % 1
            assert min(d, 1 - d) <= 2.0 ** -33.9, (p, x)


def test_far_frequencies(va):
    """Past 2^20 radians a position the two doubles run out slowly: 2^-103 of f / 2 pi and one unit."""
    f = [2.0 ** e * 1.7 for e in range(20, 64, 3)]
    turns = va.varlen_attn_rotary_turns(f)[1]
    for x, t in zip(f, turns):
        assert _off(x, t) <= 1 + x / 6.28 * 2.0 ** (64 - 103)
    assert va.varlen_attn_rotary_turns([1.7e308, -1.7e308])[0] == 0
