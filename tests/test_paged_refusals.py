"""Refusals of the paged calls, without a GPU (device pointers are fake aligned
addresses)."""
import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from indexed_sparse_attention_gb300 import build as qsa_build
from indexed_sparse_attention_gb300 import paged

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    qsa_build.build()
    return qsa.lib()


def test_extend_step_checks(L):
    pool = paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 16)
    call = lambda p=pool, seqs=FAKE, new=FAKE, n=1, to=FAKE: L.qsa_pages_extend_step(p, seqs, new, n, to, None)
    assert call(to=None) == 1 and call(to=None, n=0) == 1
    assert call(seqs=None) == 1 and call(new=None) == 1 and call(n=-1) == 1 and call(n=1025) == 2
    assert call(p=None) == 1 and call(p=paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 20)) == 2
    assert "qsa_pages_extend_step" in L.qsa_last_error().decode()


def test_pages_of_more_pieces_than_32_bits_count(L):
    # 1,024 tokens of 32,768 heads of 1,024 bytes: 2^31 pieces of 16 bytes.
    def calls(heads):
        cache = paged.PagedCacheDesc(FAKE, FAKE, 1 << 36, 256, 1 << 25, None, 0, 0, 0, 10, 1024)
        cfg = qsa.AttnConfig(heads, heads, 256, qsa.F32, qsa.F32, qsa.F32, 0.0, 0)
        pool = paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 1024)
        return (L.qsa_pages_fork(pool, cache, 1, cfg, FAKE, FAKE, None, 1, None, 0, None),
                L.qsa_pages_compact(pool, cache, 1, cfg, None, None, 0, None),
                L.qsa_pages_copy(cache, 1, cfg, None, FAKE, 1, None))
    assert calls(32768) == (2, 2, 2) and calls(65535) == (2, 2, 2)
    assert calls(32767) == (4, 4, 1)                            # only the workspace, or the list, is missing


def test_configurations_and_workspaces_of_other_calls():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache, batch = qsa.PagedCache(k, k.clone()), qsa.PagedBatch(i32(2, 4), i32(2), i32(3), n_rows=2)
    q = torch.zeros(2, 24, 128, dtype=torch.bfloat16)
    for cfg in (cache.config(32, q.dtype), cache.config(24, torch.float32),
                qsa.PagedCache(k.float(), k.float()).config(24, q.dtype),
                qsa.PagedCache(k[:, :1], k[:, :1]).config(24, q.dtype),
                qsa.PagedCache(k.view(4, 2, 8, 256), k.view(4, 2, 8, 256)).config(24, q.dtype)):
        with pytest.raises(ValueError, match="another call"):
            qsa.paged_attn(cache, batch, q, q.clone(), cfg=cfg)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8, device="meta"), torch.empty(1 << 20),
               torch.empty(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            qsa.paged_attn(cache, batch, q, q.clone(), workspace=ws)


def test_tensors_that_are_not_on_a_gpu():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache, batch = qsa.PagedCache(k, k.clone()), qsa.PagedBatch(i32(2, 4), i32(2), i32(3), n_rows=2)
    q, new = torch.zeros(2, 24, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    pool = qsa.PagePool.empty(2, 4, [cache])
    for call in (lambda: qsa.paged_attn(cache, batch, q, q.clone(), workspace=torch.empty(64, dtype=torch.uint8), stream=7),
                 lambda: qsa.paged_append(cache, batch, new, new, stream=7),
                 lambda: pool.extend(i32(1), i32(1), stream=7), lambda: pool.fork(i32(1), i32(1), stream=7),
                 lambda: pool.free(i32(1), stream=7), lambda: pool.compact(stream=7),
                 lambda: pool.copy(i32(1), i32(1), stream=7)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
