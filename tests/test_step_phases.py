"""The phases of a rotary descriptor against 1 / 2 pi to 300 bits."""
from fractions import Fraction

import pytest

import affix_kv_cache_gb300 as ac


def _arctan_of_one_over(x, one):
    term, total, n, sign = one // x, one // x, 1, 1
    while term:
        term //= x * x
        n, sign = n + 2, -sign
        total += sign * (term // n)
    return total


ONE = 1 << 330
TWO_PI = Fraction(8 * (4 * _arctan_of_one_over(5, ONE) - _arctan_of_one_over(239, ONE)), ONE)        # Machin's formula


def _off(phase, f):
    """How far a phase lies from f / 2 pi modulo one turn, in units of 2^-64 turns."""
    turns = Fraction(f) / TWO_PI
    d = (Fraction(phase) - turns * 2 ** 64) % 2 ** 64
    return min(d, 2 ** 64 - d)


@pytest.mark.parametrize("theta", [1e4, 5e5, 1e6, 10.0])
@pytest.mark.parametrize("rd", [128, 64, 36])
def test_phases_are_the_nearest(theta, rd):
    """A unit is 2^-64 turns, so that the furthest position, 2^31, is off by at most 2^-34 turns."""
    f = [theta ** (-2 * i / rd) for i in range(rd // 2)]
    r = ac.rope_desc_frequencies(f)
    assert max(_off(r.phase[i], x) for i, x in enumerate(f)) <= Fraction(1, 2) + Fraction(1, 1 << 20)
    s = ac.rope_desc(rd, theta)
    # the library's own powers may lie one step of a double beside these
    assert max(_off(s.phase[i], x) for i, x in enumerate(f)) <= 2 ** 12


def test_phases_of_any_frequency_below_a_turn():
    f = [0.0, 1.0, -1.0, 6.283185307179586, 6.2831853071795855, -6.2831853071795855, 3.0, -0.25, 1e-19, -1e-19, 2.0 ** -64, 5e-324, -5e-324, 1e-300, 6.28,
         -3.141592653589793, 0.3333333333333333]
    r = ac.rope_desc_frequencies(f)
    for i, x in enumerate(f):
        # (2 pi rounded to a double is a whole turn: its quotient is taken in double)
        assert _off(r.phase[i], x) <= (2 ** 12 if x == 6.283185307179586 else Fraction(1, 2) + Fraction(1, 1 << 20)), x
