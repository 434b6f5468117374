"""Frequencies scaled by parts, against the definition in 50 decimal digits."""
import math
from decimal import Decimal, getcontext

import pytest

import indexed_sparse_attention_gb300 as qsa

PI = Decimal("3.14159265358979323846264338327950288419716939937510582")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()


def by_turns(rot, base, factor, original, fast, slow):
    """(w, w', g) of each pair: the ramp is linear in how often the pair turns over `original` tokens."""
    getcontext().prec = 50
    f, lo, hi = (Decimal(x) for x in (factor, slow, fast))
    for i in range(rot // 2):
        w = (Decimal(base).ln() * (Decimal(-2 * i) / rot)).exp()
        g = min(Decimal(1), max(Decimal(0), (Decimal(original) * w / (2 * PI) - lo) / (hi - lo)))
        yield w, (1 - g) * w / f + g * w, g


@pytest.mark.parametrize("rot,base,factor,original,fast,slow", [
    (128, 1e6, 4.0, 32768, 32.0, 1.0), (128, 1e4, 40.0, 4096, 32.0, 1.0), (64, 5e5, 8.0, 8192, 4.0, 1.0),
    (256, 1e6, 32.0, 8192, 32.0, 0.0), (16, 1e4, 1.0, 100, 2.5, 0.25)])
def test_the_ramp_is_linear_in_turns(rot, base, factor, original, fast, slow):
    # In binary64 w is off by 2 units of 2^-53 of itself (its power), r by two more and so g by 4.2 r / (fast - slow)
    # <= 4.2 (1 + slow / (fast - slow)) of them and three of its own arithmetic; w' = w ((1 - g) / factor + g), three
    # operations on terms up to w, by 2 + g's + 3 units of w: 16 at most.
    got = qsa.Rope(rot, base=base, scaling=qsa.RopeScaling("parts", factor, original_tokens=original, fast=fast, slow=slow))
    inside = 0
    for a, (w, want, g) in zip(got.frequencies, by_turns(rot, base, factor, original, fast, slow)):
        assert abs(Decimal(a) - want) <= 16 * w / (1 << 53)
        inside += 0 < g < 1
    assert inside >= 2 and len(got.frequencies) == rot // 2
    assert math.isclose(got.magnitude, 0.1 * math.log(factor) + 1, rel_tol=2.0 ** -23)


def by_index(rot, base, factor, original, fast, slow):
    """Frequencies whose ramp is linear in the pair's index, as README works them out."""
    index = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    keep = [1 - min(max((i - a) / max(b - a, 1e-3), 0), 1) for i in range(rot // 2)]
    w = [base ** (-2 * i / rot) for i in range(rot // 2)]
    return [(1 - k) * x / factor + k * x for x, k in zip(w, keep)]


def test_a_ramp_by_index_is_another_one_and_can_be_given():
    args = (128, 1e6, 4.0, 32768, 32.0, 1.0)
    given = by_index(*args)
    own = qsa.Rope(128, base=1e6, scaling=qsa.RopeScaling("parts", 4.0, original_tokens=32768)).frequencies
    ratio = [a / b for a, b in zip(given, own)]
    same = [i for i, r in enumerate(ratio) if abs(r - 1) < 1e-12]
    # Both leave the pairs before the ramp and divide those behind it; inside they are different frequencies.
    assert set(range(24)) <= set(same) and set(range(40, 64)) <= set(same) and 1.7 < max(ratio) < 1.75 and len(same) < 50
    rope = qsa.Rope(128, frequencies=given, magnitude=0.1 * math.log(4.0) + 1)
    assert rope.frequencies == tuple(given) and math.isclose(rope.magnitude, 1.1386294, rel_tol=1e-6)
