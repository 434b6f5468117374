"""Attention over 4-bit caches where logits lie far from zero."""
import math

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import U, dev
from q4_cases import make_paged4

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


def one_key(x):
    """(index and value of the token with the largest logit, logit, what it is above the next one) of every row and head."""
    K, V = x.seq_kv(0)
    n, r, Hkv, D = x.lens[0], x.rows[0], x.k.shape[1], x.q.shape[2]
    q = x.q.double().view(r, Hkv, -1, D)
    z = torch.einsum("rhgd,htd->rhgt", q, K) * D ** -0.5
    z = z.masked_fill((torch.arange(n)[None] > torch.arange(n - r, n)[:, None])[:, None, None], -math.inf)
    two = z.topk(2, -1)
    v = torch.stack([V[h][two.indices[:, h, :, 0]] for h in range(Hkv)], 1)
    mag = (torch.einsum("rhgd,htd->rhgt", q.abs(), K.abs()) * D ** -0.5).amax(-1)
    return v.flatten(1, 2), two.values[..., 0].flatten(1, 2), (two.values[..., 0] - two.values[..., 1]).flatten(1, 2), mag.flatten(1, 2)


@pytest.mark.parametrize("D,rows", [(128, 1), (256, 1), (128, 3), (256, 3), (128, 40), (256, 5)])
@pytest.mark.parametrize("splits", [1, 0])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 19, 2.0 ** 21, 2.0 ** 23, 2.0 ** 27, 2.0 ** 40, 2.0 ** 80])
def test_logits_far_from_zero(D, rows, splits, size):
    """Logits of up to 2^83: where the largest is above the next one by more than rounding, and than log(2^26) (the
    others' weights are below 2^-26 then), the output is its V, rounded to f16, and lse that logit."""
    x = make_paged4([1500], [rows], D=D, Hkv=1, G=5, page=64, seed=19)
    x.q = (x.q.float() * size).bfloat16()
    v, z, gap, mag = one_key(x)
    # K rounded to f16 (more than 16 entries: 2^-11 of it), sums in binary32 as q4_cases has them, exponents of base 2.
    off = 2 * mag * ((2 * D + 4 * (D // 32) + 24) * U + 2.0 ** -21 + (1.01 * 2.0 ** -11 if 5 * rows > 16 else 0.0))
    sure = gap > off + 26 * math.log(2)
    assert sure.float().mean() > (0.25 if 5 * rows > 16 else 0.9) or size < 2.0 ** 19
    out, lse = (t.double().cpu() for t in run(x, n_splits=splits))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # V and the weight to f16 (the sum that divides is of unrounded weights), the output's two roundings; 1,500 other
    # tokens of weights below 2^-26.
    tol = (2.0 ** -10 * 1.01 + 4 * U) * v.abs() + 2.0 ** -25 + 1500 * 2.0 ** -26 * 2 * x.seq_kv(0)[1].abs().max()
    assert ((out - v).abs() <= tol)[sure].all()
    assert ((lse - z).abs() <= off / 2 + 8 * U * z.abs() + 1500 * 2.0 ** -26)[sure].all()
    # Whatever it is, an output lies within V's values.
    lo, hi = (getattr(x.seq_kv(0)[1], f)(1)[:, None].repeat_interleave(5, 1).transpose(0, 1).reshape(1, 5, D) for f in ("amin", "amax"))
    slack = 2.0 ** -9 * torch.maximum(lo.abs(), hi.abs())
    assert ((out >= lo - slack) & (out <= hi + slack)).all()
    assert qsa.check_device_status() == (0, "")


def test_logits_that_climb_far_from_zero():
    # Each tile's logits are above the last one's by some thousands, from minus 2^27 to plus 2^27: the last tile's are left.
    for rows, D in ((1, 256), (4, 128), (9, 128), (8, 256)):
        x = make_paged4([1500], [rows], D=D, Hkv=1, G=3, page=64, seed=18, lean=0.0)
        x.q[:] = 0.0
        x.q[..., 0] = 2.0 ** 20
        for t in range(1500):
            # (minima of f16's integers: exact)
            records(x)[x.table[0, t // 64], 0, t % 64, 0, 0] = torch.tensor([0.0, float(t - 750)], dtype=torch.float16)
        out, lse = run(x)
        V = x.seq_kv(0)[1][0]
        want = V[1500 - rows:][:, None].expand(-1, 3, -1)
        assert ((out.double().cpu() - want).abs() <= (2.0 ** -10 * 1.01 + 4 * U) * want.abs() + 2.0 ** -25).all()
        z = (torch.arange(1500 - rows, 1500) - 750).double()[:, None] * 2.0 ** 20 * D ** -0.5
        assert ((lse.double().cpu() - z).abs() <= 8 * U * z).all()
