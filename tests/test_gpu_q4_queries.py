"""Attention of queries with channels far above the others over 4-bit caches.

Tolerances are those of q4_cases, with q's part as the header states it.  Up to 16 entries q is the sum of an E5M2 and
an E4M3 code of it times a power of two that brings the row's largest magnitude qmax to [2^11, 2^12).  A value v of
[2^e, 2^(e + 1)) leaves at most 2^(e - 3) behind its E5M2 code (3 significant bits), which is at most 16 of bf16's units
2^(e - 7), so that E4M3's 4 bits hold it where the unit is a step of E4M3 (2^-9): for e >= -2, values from 2^-13 qmax on.
Smaller ones are off by half of that step, dq <= min(2^-21 qmax, |q|): logits by up to max_t scale sum_c dq_c |k_tc|."""
import math

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import U, assert_attended, dev
from q4_cases import attend4, make_paged4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    qsa.check_device_status()


def run(x, **kw):
    cache, batch, q = x.device()
    out, lse = torch.full(q.shape, 7.0, device=dev()), torch.full(q.shape[:2], 7.0, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def records(x):
    """x's scales and minima: [n_pages, Hkv, page, K or V, block, scale or minimum]."""
    return x.scale.view(*x.scale.shape[:3], 2, -1, 2)


def narrow_tolerances(x, scale=None):
    """(out, lse, tolerances) of a call of up to 16 entries, with the header's bound of q."""
    out, lse, _, _ = attend4(x, scale=scale)
    D, Hkv = x.q.shape[2], x.k.shape[1]
    G, scale = x.q.shape[1] // Hkv, scale or D ** -0.5
    otol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for i, (n, r) in enumerate(zip(x.lens, x.rows)):
        K, V = x.seq_parts(i)
        r0 = int(x.row_start[i])
        see = torch.arange(n)[None] <= torch.arange(n - r, n)[:, None]
        for h in range(Hkv):
            kmag, v = (K[0][h] * K[1][h]).abs() + K[2][h].abs(), V[0][h] * V[1][h] + V[2][h]
            q = x.q[r0:r0 + r, h * G:(h + 1) * G].double()
            top = q.abs().amax(-1, keepdim=True)
            dq = torch.where(q.abs() < 2.0 ** -13 * top, torch.minimum(q.abs(), 2.0 ** -21 * top), 0.0)
            mag, lost = ((torch.einsum("rgd,td->rgt", y, kmag) * scale).masked_fill(~see[:, None], 0.0).amax(-1) for y in (q.abs(), dq))
            e = 2 * ((2 * D + 4 * (D // 32) + 24) * U * mag + lost) + 8 * U
            k = K[0][h] * K[1][h] + K[2][h]
            z = (torch.einsum("rgd,td->rgt", q, k) * scale).masked_fill(~see[:, None], -math.inf)
            wabs = torch.einsum("rgt,td->rgd", z.softmax(-1), v.abs())
            cnt, sl = see.sum(1)[:, None].double(), slice(h * G, (h + 1) * G)
            rounded = 1.01 * 2.0 ** -10 * wabs + 2.0 ** -25 + cnt[..., None] * 2.0 ** -32 * v.abs().max()
            otol[r0:r0 + r, sl] = (2 * (e + (cnt + 16) * 2 * U))[..., None] * wabs + rounded
            ltol[r0:r0 + r, sl] = e + (cnt + 16) * 2 * U + 4 * U * lse[r0:r0 + r, sl].abs()
    return out, lse, otol, ltol


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("times", [150, 1000, 4000])
def test_queries_with_channels_far_above_the_others(D, times):
    # One block of q's channels is larger, and the keys' scale and minimum of it smaller by as much, so that all
    # channels matter to the logits.
    x = make_paged4([900, 130], [1, 3], D=D, page=32, Hkv=2, G=4, seed=67)
    x.q[..., :32] *= times
    records(x)[..., 0, 0, :] = (records(x)[..., 0, 0, :].float() / times).half()
    out, lse = run(x)
    assert_attended(out, lse, narrow_tolerances(x))
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("below", [9, 10, 11, 12, 13])
def test_small_channels_of_a_query_are_exact(D, below):
    # All channels but the first block's are one value of 2^-below of the largest, another of bf16's values for each head,
    # and the keys, positive, are zero in the first block: what such a value loses adds up over all channels.
    x = make_paged4([200, 33], [1, 3], D=D, page=16, Hkv=1, G=5, seed=69)
    heads = (1 + torch.tensor([1, 37, 64 + 11, 64 + 33, 127]) / 128) * 2.0 ** -below
    x.q = heads[None, :, None].expand(4, 5, D).bfloat16().contiguous()
    x.q[..., :32] = 1.0 + torch.arange(32) / 128
    x.q *= 2.0 ** torch.tensor([0.0, 5.0, 9.0, -40.0])[:, None, None]
    rec = records(x)[..., 0, :, :]
    rec[..., 1] = 0.0
    rec[..., 0, 0] = 0.0
    rec[..., 1:, 0] = rec[..., 1:, 0].abs()
    for scale in (None, 2.0 ** -50):
        out, lse = run(x, scale=scale or 0.0)
        assert_attended(out, lse, narrow_tolerances(x, scale))
