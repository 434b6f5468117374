"""4-bit caches with pages smaller and larger than the boxes that a call of more than 16 entries copies them in, and
with pages that are missing."""
import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import assert_attended, dev
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


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("D", [128, 256])
def test_page_sizes_of_many_entries(page, order, D):
    x = make_paged4([1500, 3, 129, 2100], [4, 2, 9, 40], D=D, page=page, order=order, seed=page, poison=True)
    for window, sinks in ((0, 0), (300, 20), (700, 200)):
        out, lse = run(x, window=window, n_sinks=sinks)
        assert_attended(out, lse, attend4(x, window, sinks))
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("page", [16, 32, 128, 512])
@pytest.mark.parametrize("rows", [[1, 1], [2, 5]])
def test_missing_pages_of_every_size(D, page, rows):
    # Pages 1 and 3 of the first sequence and 2 of the second are not there: their tokens are skipped, and counted.
    x = make_paged4([4 * page + 7, 3 * page], rows, D=D, page=page, seed=11, poison=True)
    full = x.table.clone()
    x.table[0, 1], x.table[0, 3], x.table[1, 2] = -1, 1 << 20, x.k.shape[0]
    out, lse = run(x)
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "page table entries" in why
    x.table = full
    for i, gone in ((0, {1, 3}), (1, {2})):
        K, V = x.seq_kv(i)
        r0, n, r = int(x.row_start[i]), x.lens[i], x.rows[i]
        for j in range(r):
            see = torch.tensor([t <= n - r + j and t // page not in gone for t in range(n)])
            for h in range(2):
                z = (x.q[r0 + j, 12 * h:12 * h + 12].double() @ K[h].T) * D ** -0.5
                z = z.masked_fill(~see, float("-inf"))
                # As in q4_cases: V, the weights and (2 and 5 rows) K rounded to f16, heads' q up to 3 sqrt(D) long.
                k_off = 2.0 ** -11 * 1.01 * (x.q[r0 + j, 12 * h:12 * h + 12].double().abs() @ K[h].abs().T).amax() * D ** -0.5
                tol = (2 * k_off + 2.0 ** -10 * 1.01 + 2.0 ** -12) * V[h][see].abs().max()
                assert (out[r0 + j, 12 * h:12 * h + 12].double().cpu() - torch.softmax(z, -1) @ V[h]).abs().max() < tol
                assert (lse[r0 + j, 12 * h:12 * h + 12].double().cpu() - torch.logsumexp(z, -1)).abs().max() < 2 * k_off + 2.0 ** -12
