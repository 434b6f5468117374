"""The paged-cache entry points without a GPU: every check of their arguments
runs on the host before a launch.  Device pointers are fake aligned addresses."""
import ctypes

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from indexed_sparse_attention_gb300 import build as qsa_build
from indexed_sparse_attention_gb300 import paged

FAKE, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    qsa_build.build()
    return qsa.lib()


def _cache(**kw):
    c = paged.PagedCacheDesc(FAKE, FAKE, 2 * 16 * 128, 16 * 128, 128, None, 0, 0, 0, 10, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _fp8(**kw):
    return _cache(**{"kv_scale": FAKE, "scale_page_stride": 32, "scale_head_stride": 16, "scale_tok_stride": 1, **kw})


def _batch(**kw):
    b = paged.PagedBatchDesc(FAKE, 8, FAKE, FAKE, 2, 3, 2)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _cfg(**kw):
    c = qsa.AttnConfig(24, 2, 128, qsa.BF16, qsa.BF16, qsa.F32, 0.0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


FP8 = {"kv_dtype": qsa.FP8}
CACHES = [(2, {"page_tokens": 24}, {}), (2, {"page_tokens": 8}, {}), (2, {"page_tokens": 2048}, {}),
          (1, {"n_pages": 0}, {}), (1, {"k": None}, {}), (1, {"tok_stride": 64}, {}), (1, {"head_stride": 0}, {}),
          (1, {"page_stride": -4096}, {}), (3, {"v": MIS}, {}), (3, {"tok_stride": 132}, {}),
          (3, {"page_stride": 4100}, {}), (1, {}, FP8), (2, {}, {"kv_dtype": qsa.Q8}), (2, {}, {"kv_dtype": 9}),
          (2, {}, {"head_dim": 64}), (2, {}, {"q_dtype": qsa.F32}), (2, {}, {"n_q_heads": 34}),
          (1, {}, {"n_q_heads": 25}), (1, {}, {"n_splits": -1}), (1, {}, {"scale": -1.0})]


@pytest.mark.parametrize("want,cache,cfg", CACHES)
def test_cache_and_config_checks(L, want, cache, cfg):
    c, b, g = _cache(**cache), _batch(), _cfg(**cfg)
    at = L.qsa_paged_attn(c, b, g, 0, 0, FAKE, FAKE, FAKE, FAKE, 1 << 40, None)
    assert at == want and "qsa_paged_attn" in L.qsa_last_error().decode()
    assert L.qsa_paged_append(c, b, g, FAKE, FAKE, 256, 128, None) == want
    pool = paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 16)
    assert L.qsa_pages_fork(pool, c, 1, g, FAKE, FAKE, None, 2, FAKE, 1 << 40, None) == want
    assert L.qsa_pages_compact(pool, c, 1, g, None, FAKE, 1 << 40, None) == want
    assert L.qsa_pages_copy(c, 1, g, FAKE, FAKE, 2, None) == want


def test_attention_checks(L):
    c, g = _cache(), _cfg()
    call = lambda b=_batch(), w=0, s=0, q=FAKE, out=FAKE, ws=FAKE, n=1 << 40: L.qsa_paged_attn(
        c, b, g, w, s, q, out, None, ws, n, None)
    assert call(w=-1) == 1 and call(s=-1) == 1
    assert call(q=None) == 1 and call(out=None) == 1
    assert call(q=MIS) == 3 and call(out=MIS) == 3 and call(ws=MIS) == 3
    assert call(_batch(table=None)) == 1 and call(_batch(lens=None)) == 1 and call(_batch(row_start=None)) == 1
    assert call(_batch(table_ld=0)) == 1 and call(_batch(n_seqs=-1)) == 1 and call(_batch(n_rows=-1)) == 1
    assert call(_batch(n_rows=1 << 30)) == 2
    need = L.qsa_paged_attn_workspace_size(_batch(), g)
    assert need > 0
    assert call(n=need - 1) == 4 and call(ws=None) == 4
    assert call(_batch(n_rows=0), q=None, out=None, ws=None, n=0) == 0        # nothing to do
    assert call(_batch(n_seqs=0), q=None, out=None, ws=None, n=0) == 0
    assert L.qsa_paged_attn(None, _batch(), g, 0, 0, FAKE, FAKE, None, FAKE, need, None) == 1
    assert L.qsa_paged_attn(c, None, g, 0, 0, FAKE, FAKE, None, FAKE, need, None) == 1
    assert L.qsa_paged_attn(c, _batch(), None, 0, 0, FAKE, FAKE, None, FAKE, need, None) == 1
    # The workspace follows the shape of the call, not the lengths; fewer runs need less.
    one = _cfg(n_splits=1)
    assert L.qsa_paged_attn_workspace_size(_batch(), one) < need
    assert L.qsa_paged_attn_workspace_size(_batch(), _cfg(head_dim=64)) == 0


def test_fp8_scale_checks(L):
    g = _cfg(**FP8)
    call = lambda c: L.qsa_paged_attn(c, _batch(), g, 0, 0, FAKE, FAKE, None, None, 0, None)
    assert call(_fp8(kv_scale=0x10002)) == 3
    assert call(_fp8(scale_tok_stride=0)) == 1
    assert call(_fp8()) == 4                                                 # only the workspace is missing


def test_append_checks(L):
    call = lambda k=FAKE, v=FAKE, rs=256, hs=128, b=_batch(): L.qsa_paged_append(_cache(), b, _cfg(), k, v, rs, hs, None)
    assert call(k=None) == 1 and call(v=None) == 1
    assert call(k=MIS) == 3 and call(rs=260) == 3 and call(hs=132) == 3
    assert call(rs=-256) == 1 and call(hs=-128) == 1
    assert call(b=_batch(n_rows=0), k=None) == 0


def test_page_call_checks(L):
    pool = lambda **kw: paged.PagePoolDesc(**{"table": FAKE, "table_ld": 8, "lens": FAKE, "refs": FAKE, "n_seqs": 4,
                                              "n_pages": 10, "page_tokens": 16, **kw})
    for want, kw in [(1, {"n_seqs": 0}), (1, {"n_pages": 0}), (1, {"table_ld": 0}), (2, {"page_tokens": 20}),
                     (2, {"n_pages": (1 << 24) + 1}), (1, {"table": None}), (1, {"refs": None})]:
        p = pool(**kw)
        assert L.qsa_pages_workspace_size(p) == 0
        assert L.qsa_pages_extend(p, FAKE, FAKE, 1, None) == want
        assert L.qsa_pages_free(p, FAKE, None, 1, None) == want
        assert L.qsa_pages_fork(p, None, 0, None, FAKE, FAKE, None, 1, FAKE, 1 << 30, None) == want
        assert L.qsa_pages_compact(p, None, 0, None, None, FAKE, 1 << 30, None) == want
    p = pool()
    need = L.qsa_pages_workspace_size(p)
    assert need > 0
    assert L.qsa_pages_extend(p, None, FAKE, 1, None) == 1 and L.qsa_pages_extend(p, FAKE, None, 1, None) == 1
    assert L.qsa_pages_extend(p, FAKE, FAKE, 1025, None) == 2 and L.qsa_pages_extend(p, FAKE, FAKE, -1, None) == 1
    assert L.qsa_pages_extend(p, None, None, 0, None) == 0
    assert L.qsa_pages_free(p, None, None, 1, None) == 1 and L.qsa_pages_free(p, None, None, 0, None) == 0
    c, g = _cache(), _cfg()
    fork = lambda caches=c, n=1, src=FAKE, dst=FAKE, m=1, ws=FAKE, size=need: L.qsa_pages_fork(
        p, caches, n, g, src, dst, None, m, ws, size, None)
    assert fork(n=257) == 2 and fork(n=-1) == 2 and fork(caches=None) == 1
    assert fork(src=None) == 1 and fork(dst=None) == 1 and fork(m=1025) == 2
    assert fork(size=need - 1) == 4 and fork(ws=None) == 4 and fork(ws=MIS) == 3
    assert fork(m=0, src=None, dst=None) == 0
    assert fork(caches=_cache(n_pages=9)) == 1                               # fewer pages than the pool counts
    assert fork(caches=_cache(page_tokens=32)) == 1
    assert L.qsa_pages_compact(p, c, 1, g, None, FAKE, need - 1, None) == 4
    copy = lambda caches=c, src=FAKE, dst=FAKE, n=2: L.qsa_pages_copy(caches, 1, g, src, dst, n, None)
    assert copy(src=None) == 1 and copy(dst=None) == 1 and copy(n=-1) == 1 and copy(n=0, src=None) == 0


def test_python_refusals():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qsa.PagedCache(k, k[:2])
    with pytest.raises(TypeError):
        qsa.PagedCache(k.transpose(2, 3), k.transpose(2, 3))                 # channels not unit stride
    with pytest.raises(ValueError):
        qsa.PagedCache(k, k, kv_scale=torch.zeros(4, 2, 16, 2, dtype=torch.float16))
    c8 = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    with pytest.raises(ValueError):
        qsa.PagedCache(c8, c8)
    with pytest.raises(TypeError):
        qsa.PagedCache(c8, c8, kv_scale=torch.zeros(4, 2, 16, 2))
    cache = qsa.PagedCache(k, k.clone())
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(TypeError):
        qsa.PagedBatch(i32(2, 4).long(), i32(2), i32(3), n_rows=2)
    with pytest.raises(ValueError):
        qsa.PagedBatch(i32(2, 4), i32(2), i32(2), n_rows=2)
    with pytest.raises(TypeError):
        qsa.PagedBatch(i32(2, 8)[:, :4], i32(2), i32(3), n_rows=2)           # rows of a wider table
    batch = qsa.PagedBatch(i32(2, 4), i32(2), i32(3), n_rows=2)
    q = torch.zeros(2, 24, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be"):
        qsa.paged_attn(cache, batch, q[:1], q[:1].clone())
    with pytest.raises(ValueError, match="q must be"):
        qsa.paged_attn(cache, batch, q.float(), q.float())
    with pytest.raises(ValueError, match="out must be"):
        qsa.paged_attn(cache, batch, q, q[:, :12].clone())
    with pytest.raises(ValueError, match="contiguous"):
        qsa.paged_attn(cache, batch, torch.zeros(2, 48, 128, dtype=torch.bfloat16)[:, ::2], q)
    with pytest.raises(ValueError, match="k_new must be"):
        qsa.paged_append(cache, batch, k[0, :, :1], k[0, :, :1])
    with pytest.raises(ValueError, match="equal strides"):
        rows = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
        qsa.paged_append(cache, batch, rows, torch.zeros(2, 4, 128, dtype=torch.bfloat16)[:, :2])
