"""The 64-bit turns of a rotation, against 50 digits."""
from fractions import Fraction

import pytest

import indexed_sparse_attention_gb300 as qsa

PI = Fraction("3.14159265358979323846264338327950288419716939937510582")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()


def test_frequencies_of_any_size_make_a_rotation():
    # (Beyond 2^52 turns a position there is no fraction left to speak of.)
    for w in (1e16, 1e30, 1e200, 1.7976931348623157e308):
        a, b = (qsa.Rope(16, frequencies=[x] * 8).desc.turns[0] for x in (w, -w))
        assert (a + b) % (1 << 64) == 0


def test_turns_are_the_nearest_64_bits():
    # w / (2 pi) of the binary64 w, modulo 1: off by half of 2^-64 of a turn, and by the 2^-52 of it that remain of a
    # quotient of two binary64 numbers each (2^-104 of the turns: nothing beside it, up to 2^40 radians).
    ws = [1.0, 0.3, 1e-6, 3.14159, 0.0, 7.5, 1e6 ** (-254 / 256) / 32, 2.0 ** -60, 6.283185307179586, 1e5, 2.0 ** 40, 1e-300, 5e-324]
    for w in ws + [-w for w in ws]:
        t = qsa.Rope(16, frequencies=[w] * 8).desc.turns[0]
        exact = Fraction(w) / (2 * PI) * (1 << 64)
        off = (Fraction(t) - exact) % (1 << 64)
        off = min(off, (1 << 64) - off)
        assert off <= Fraction(1, 2) + Fraction(1, 1 << 10), (w, float(off))
    for w in ws:   # opposite frequencies are opposite turns
        plus, minus = (qsa.Rope(16, frequencies=[x] * 8).desc.turns[0] for x in (w, -w))
        assert (plus + minus) % (1 << 64) == 0
