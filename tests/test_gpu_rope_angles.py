"""Rotations by small angles, whose sine is as exact as the values are, and by opposite ones."""
import math

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import U, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")


def turn_ones(rope, pos):
    """(cos, sin) of every pair and position: pairs (1, 0), turned; [positions, pairs]."""
    R = rope.rot_dim
    x = torch.zeros(len(pos), 1, R, device=dev())
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if rope.pairs else (i, i + R // 2)
    x[..., a] = 1.0
    got = qsa.rotate(rope, torch.tensor(pos, dtype=torch.int32, device=dev()), x)[:, 0].double().cpu()
    return got[:, a], got[:, b]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("scaling", [None, qsa.RopeScaling("linear", 32.0), qsa.RopeScaling("parts", 32.0, original_tokens=8192)])
def test_sines_of_small_angles(pairs, scaling):
    # An angle p w below pi / 4: turns off by 2^-65 of a turn for each position; rounded to binary32, U of itself, which
    # a sine passes on at most as it is; sincospi within 2 units (4 U); the cosine's and the magnitude's products are
    # exact but for one rounding, U.  The reference's own w and products are binary64.
    rope = qsa.Rope(256, base=1e6, pairs=pairs, scaling=scaling, magnitude=1.0)
    pos = [1, -1, 2, 3, 7, -100, 1000, 65_537, -1_000_003, 2 ** 31 - 1]
    cos, sin = turn_ones(rope, pos)
    angle = torch.tensor(pos, dtype=torch.float64)[:, None] * torch.tensor(rope.frequencies, dtype=torch.float64)
    small = angle.abs() < math.pi / 4
    assert small[0].sum() > 100 and small.any(1).sum() >= 8
    tol = 8 * U * angle.sin().abs() + angle.abs() * 2.0 ** -51 + torch.tensor(pos).abs()[:, None] * (2 * math.pi * 2.0 ** -65)
    err = (sin - angle.sin()).abs()
    assert (err <= tol)[small].all(), f"worst {float((err / tol)[small].max()):.3g} of its tolerance"
    assert ((cos - angle.cos()).abs() <= 8 * U)[small].all()


@pytest.mark.parametrize("pairs", [False, True])
def test_opposite_positions_turn_by_opposite_angles(pairs):
    rope = qsa.Rope(128, base=1e6, pairs=pairs, scaling=qsa.RopeScaling("linear", 3.0))
    g = torch.Generator().manual_seed(1)
    pos = [1, 2, 3] + torch.randint(1, 2 ** 31 - 1, (400,), generator=g).tolist()
    (c0, s0), (c1, s1) = turn_ones(rope, pos), turn_ones(rope, [-p for p in pos])
    assert torch.equal(c0, c1) and torch.equal(s0, -s1)
