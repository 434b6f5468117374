"""Paged attention of batches of more sequences than a warp divides by itself, with
prompts among single rows."""
import random

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import assert_attended, attend64, dev, make_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    qsa.check_device_status()


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("n,chunks", [(65, {64: 300}), (65, {0: 300}), (130, {129: 290, 70: 9}), (300, {299: 310}),
                                      (420, {3: 280, 200: 37, 401: 300, 419: 5})])
def test_prompts_in_large_batches(dtype, n, chunks):
    rng = random.Random(n)
    lens = [rng.randint(1, 60) for _ in range(n)]
    rows = [1 if rng.random() < 0.9 else 0 for _ in range(n)]
    for i, r in chunks.items():
        lens[i], rows[i] = r + rng.randint(0, 200), r
    x = make_paged(lens, rows, dtype=dtype, D=128, Hkv=1, G=4, page=16, seed=n, poison=True)
    cache, batch, q = x.device()
    out, lse = torch.full(q.shape, 7.0, device=dev()), torch.full(q.shape[:2], 7.0, device=dev())
    for window, sinks, n_splits in ((0, 0, 0), (40, 3, 0), (0, 0, 7)):
        qsa.paged_attn(cache, batch, q, out, lse, window=window, n_sinks=sinks, n_splits=n_splits)
        torch.cuda.synchronize()
        assert_attended(out, lse, attend64(x, window, sinks))
    assert qsa.check_device_status() == (0, "")
