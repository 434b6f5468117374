"""4-bit caches: what is far, infinite or no number in one row or key stays with the rows that see it."""
import math

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import dev
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
    assert qsa.check_device_status() == (0, "")
    return out.cpu(), lse.cpu()


CASES = [(128, [1, 1]), (256, [3, 1]), (128, [40, 2]), (256, [9, 30])]


@pytest.mark.parametrize("D,rows", CASES)
@pytest.mark.parametrize("size", [2.0 ** 22, 2.0 ** 30, 2.0 ** 60])
def test_a_row_of_far_logits_leaves_the_others_their_bits(D, rows, size):
    x = make_paged4([1300, 400], rows, D=D, Hkv=2, G=5, page=32, seed=71)
    good = run(x)
    far = torch.zeros(x.q.shape[:2], dtype=torch.bool)
    for r, h in ((0, 3), (sum(rows) - 1, 6), (rows[0] // 2, 9)):
        x.q[r, h] = x.q[r, h] * size
        far[r, h] = True
    out, lse = run(x)
    assert torch.equal(out[~far], good[0][~far]) and torch.equal(lse[~far], good[1][~far])
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    again = run(x)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("D,rows", CASES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4)])
@pytest.mark.parametrize("bad", [(math.nan, 0.0), (1.0, math.nan), (0.0, math.inf), (0.0, -math.inf), (math.inf, 0.0)])
def test_a_key_that_is_no_number_stays_with_its_rows(D, rows, window, sinks, bad):
    """A block whose scale or minimum is NaN makes the logits of the rows that see it NaN; infinite ones give NaN or
    leave the key out (a logit of minus infinity)."""
    x = make_paged4([1300, 400], rows, D=D, Hkv=2, G=5, page=32, seed=72)
    good = run(x, window=window, n_sinks=sinks)
    sees = torch.zeros(x.q.shape[:2], dtype=torch.bool)
    for i, t, h in ((0, 1299 - rows[0] // 2, 0), (1, 2, 1), (1, 399 - rows[1] // 2, 0)):
        x.scale.view(*x.scale.shape[:3], 2, -1, 2)[x.table[i, t // 32], h, t % 32, 0, 1] = torch.tensor(bad, dtype=torch.float16)
        for j in range(rows[i]):
            pos = x.lens[i] - rows[i] + j
            if t <= pos and (not window or t > pos - window or t < sinks):
                sees[int(x.row_start[i]) + j, 5 * h:5 * h + 5] = True
    out, lse = run(x, window=window, n_sinks=sinks)
    assert sees.any() and not sees.all()
    assert torch.equal(out[~sees], good[0][~sees]) and torch.equal(lse[~sees], good[1][~sees])
    if any(math.isnan(b) for b in bad):
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
    else:
        whole = torch.isfinite(out).all(-1)
        assert (whole | torch.isnan(out).all(-1))[sees].all() and (torch.isfinite(lse) == whole)[sees].all()
