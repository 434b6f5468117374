"""Paged K/V caches: attention over them, their writer, and their pages
(include/qsa.h, "Paged K/V caches").  Argument marshalling only.

    pages = PagePool(table, lens, refs, caches)          # who holds which page
    batch = PagedBatch(pages.table, pages.step_lens, row_start, n_rows=R, max_rows=M)
    pages.extend(seqs, n_new)                            # room for the step's tokens, and its lengths
    step = PagedStep(caches[layer], batch, q, window=W, n_sinks=S)
    out, lse = step.run(k_new, v_new)                    # append, then attend (with rope=: rotate K and q on the way)
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Sequence

import torch

from . import AttnConfig, BF16, F32, FP8, Q4, _dtype_code, _ptr, _scratch, lib
from .calls import _call, _call_at
from .rope import Rope, RopeDesc, _strides


class PagedCacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("tok_stride", ctypes.c_int64), ("kv_scale", ctypes.c_void_p),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_tok_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32)]


class PagedBatchDesc(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_ld", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("row_start", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("max_rows", ctypes.c_int32)]


class PagePoolDesc(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_ld", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("n_seqs", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32)]


MIN_PAGE_TOKENS, MAX_PAGE_TOKENS = 16, 1024
MAX_PAGE_REQUESTS = 1024
MAX_CACHES = 256


def declare(L: ctypes.CDLL):
    """Argument types of the entry points, on the loaded library."""
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cachep, batchp, poolp, cfgp = (ctypes.POINTER(t) for t in (PagedCacheDesc, PagedBatchDesc, PagePoolDesc, AttnConfig))
    L.qsa_paged_attn_workspace_size.argtypes = [batchp, cfgp]
    L.qsa_paged_attn_workspace_size.restype = sz
    L.qsa_paged_attn.argtypes = [cachep, batchp, cfgp, i32, i32, vp, vp, vp, vp, sz, vp]
    L.qsa_paged_append.argtypes = [cachep, batchp, cfgp, vp, vp, i64, i64, vp]
    L.qsa_paged_append_rotate.argtypes = [cachep, batchp, cfgp, ctypes.POINTER(RopeDesc), vp, vp, i64, i64, vp, i64, i64, vp, vp]
    L.qsa_paged_read.argtypes = [cachep, batchp, cfgp, vp, vp, vp]
    L.qsa_pages_workspace_size.argtypes = [poolp]
    L.qsa_pages_workspace_size.restype = sz
    L.qsa_pages_extend.argtypes = [poolp, vp, vp, i32, vp]
    L.qsa_pages_extend_step.argtypes = [poolp, vp, vp, i32, vp, vp]
    L.qsa_pages_fork.argtypes = [poolp, cachep, i32, cfgp, vp, vp, vp, i32, vp, sz, vp]
    L.qsa_pages_free.argtypes = [poolp, vp, vp, i32, vp]
    L.qsa_pages_compact.argtypes = [poolp, cachep, i32, cfgp, vp, vp, sz, vp]
    L.qsa_pages_copy.argtypes = [cachep, i32, cfgp, vp, vp, i32, vp]
    for name in ("attn", "append", "append_rotate", "read"):
        getattr(L, f"qsa_paged_{name}").restype = i32
    for name in ("extend", "extend_step", "fork", "free", "compact", "copy"):
        getattr(L, f"qsa_pages_{name}").restype = i32


def _int_list(name: str, t: torch.Tensor, like: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 vector")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the pool on {like.device}")
    return t


# ---------------------------------------------------------------------- descriptions

class PagedCache:
    """One layer's cache: k, v are [n_pages, Hkv, page_tokens, D] views (channel
    stride 1, equal strides; any order of the other axes in memory).  fp8: E4M3
    codes (float8_e4m3fn or uint8) and kv_scale, an [n_pages, Hkv, page_tokens, 2]
    float16 view of the (K, V) scale pairs.  4 bits (kv_dtype=Q4): uint8 views of
    [n_pages, Hkv, page_tokens, D / 2] codes and an [n_pages, Hkv, page_tokens, D / 8]
    float16 view of the records, (scale, minimum) of K's blocks, then V's; the order of
    the codes is include/qsa.h's, and paged_append and paged_read write and read it.
    PagedCache.zeros makes a cache of any kind."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, kv_scale: torch.Tensor | None = None,
                 kv_dtype: int | None = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [n_pages, Hkv, page_tokens, D] of one shape, dtype and device")
        if k.stride(3) != 1 or k.stride() != v.stride():
            raise TypeError("k and v need unit channel stride and equal strides")
        self.k, self.v, self.kv_scale = k, v, kv_scale
        self.n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = (int(x) for x in k.shape)
        self.kv_dtype = _dtype_code(k) if kv_dtype is None else int(kv_dtype)
        q4 = self.kv_dtype == Q4
        if kv_dtype is not None and (k.dtype is not torch.uint8 if q4 else self.kv_dtype != _dtype_code(k)):
            raise TypeError(f"kv_dtype {kv_dtype} does not hold {k.dtype}")
        per = 2 if q4 else 1   # elements of a byte
        self.head_dim *= per
        d = self.desc = PagedCacheDesc()
        d.k, d.v = k.data_ptr(), v.data_ptr()
        d.page_stride, d.head_stride, d.tok_stride = (per * k.stride(i) for i in range(3))
        d.n_pages, d.page_tokens = self.n_pages, self.page_tokens
        if (kv_scale is not None) != (self.kv_dtype in (FP8, Q4)):
            raise ValueError("kv_scale goes with an fp8 or 4-bit cache")
        if kv_scale is not None:
            s = kv_scale
            n = self.head_dim // 8 if q4 else 2   # halves of a record
            if s.dtype != torch.float16 or tuple(s.shape) != (*k.shape[:3], n) or s.stride(3) != 1 or any(
                    s.stride(i) % n for i in range(3)):
                raise TypeError(f"kv_scale must be a float16 [n_pages, Hkv, page_tokens, {n}] view of whole scale records")
            if s.device != k.device:
                raise ValueError("kv_scale on another device than k")
            d.kv_scale = s.data_ptr()
            d.scale_page_stride, d.scale_head_stride, d.scale_tok_stride = (s.stride(i) // n for i in range(3))
        self.byref = ctypes.byref(d)
        self.device, self.index = k.device, k.get_device()
        self.row_dtype = torch.float32 if self.kv_dtype == F32 else torch.bfloat16   # of new rows and queries
        self._row_cfg = self.config()
        self._row_cfg_ref = ctypes.byref(self._row_cfg)
        self._read_cfg = [ctypes.byref(self.config(out_dtype=t)) for t in (torch.float32, torch.bfloat16)]
        self._rows_cfgs = {}
        self._last_call = None, None

    def _rows_cfg(self, n_q_heads: int):
        if n_q_heads not in self._rows_cfgs:
            self._rows_cfgs[n_q_heads] = ctypes.byref(self.config(n_q_heads))
        return self._rows_cfgs[n_q_heads]

    @classmethod
    def zeros(cls, n_pages: int, n_kv_heads: int, page_tokens: int, head_dim: int, kv_dtype: int = BF16,
              device="cuda") -> "PagedCache":
        """A cache of zeros, its pages' heads one after the other; kv_dtype F32, BF16, FP8 or Q4."""
        kinds = {F32: torch.float32, BF16: torch.bfloat16, FP8: torch.float8_e4m3fn, Q4: torch.uint8}
        if kv_dtype not in kinds:
            raise ValueError(f"no paged cache of kv_dtype {kv_dtype}")
        if kv_dtype == Q4 and int(head_dim) % 32:
            raise ValueError(f"4-bit rows are blocks of 32 channels, head_dim is {head_dim}")
        shape = (int(n_pages), int(n_kv_heads), int(page_tokens))
        width = int(head_dim) // 2 if kv_dtype == Q4 else int(head_dim)
        k, v = (torch.zeros(*shape, width, dtype=kinds[kv_dtype], device=device) for _ in range(2))
        record = {FP8: 2, Q4: int(head_dim) // 8}.get(kv_dtype)
        scale = None if record is None else torch.zeros(*shape, record, dtype=torch.float16, device=device)
        return cls(k, v, scale, kv_dtype)

    def config(self, n_q_heads: int | None = None, out_dtype=torch.float32, scale: float = 0.0,
               n_splits: int = 0) -> AttnConfig:
        hq = self.n_kv_heads if n_q_heads is None else int(n_q_heads)
        return AttnConfig(hq, self.n_kv_heads, self.head_dim, F32 if self.kv_dtype == F32 else BF16, self.kv_dtype,
                          F32 if out_dtype is torch.float32 else BF16 if out_dtype is torch.bfloat16
                          else _dtype_code(torch.empty(0, dtype=out_dtype)), float(scale), int(n_splits))

    def _call_config(self, n_q_heads: int, out_dtype, scale: float, n_splits: int) -> AttnConfig:
        """config() of the last call, while calls ask for the same."""
        key = (n_q_heads, out_dtype, scale, n_splits)
        last = self._last_call   # (one read: other threads may call, too)
        if last[0] != key:
            last = self._last_call = key, self.config(n_q_heads, out_dtype, scale, n_splits)
        return last[1]


class PagedBatch:
    """The sequences and rows of a call.  table [n_seqs, >= pages], lens [n_seqs]
    and row_start [n_seqs + 1] are int32 tensors on the GPU, read when the work
    runs; n_rows is the rows of q, max_rows the most that one sequence has.  Give
    max_rows: without it the call is laid out for one sequence of all rows, which
    is right for a single prompt and slower for a batch of few rows each."""

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, row_start: torch.Tensor, *, n_rows: int,
                 max_rows: int | None = None):
        if any(t.dtype != torch.int32 for t in (table, lens, row_start)):
            raise TypeError("table, lens and row_start must be int32")
        if table.dim() != 2 or not table.is_contiguous():
            raise TypeError("table must be a contiguous [n_seqs, pages]")
        n = int(table.shape[0])
        if tuple(lens.shape) != (n,) or tuple(row_start.shape) != (n + 1,) or not (
                lens.is_contiguous() and row_start.is_contiguous()):
            raise ValueError("lens must be [n_seqs] and row_start [n_seqs + 1], contiguous")
        if len({t.device for t in (table, lens, row_start)}) != 1:
            raise ValueError("table, lens and row_start on different devices")
        self.table, self.lens, self.row_start = table, lens, row_start
        self.index = table.get_device()
        self.n_seqs, self.n_rows = n, int(n_rows)
        self.max_rows = self.n_rows if max_rows is None else int(max_rows)
        ld = int(table.shape[1])
        self.desc = PagedBatchDesc(table.data_ptr(), ld, lens.data_ptr(), row_start.data_ptr(), n, self.n_rows,
                                   self.max_rows)
        self.byref = ctypes.byref(self.desc)


# Devices are compared by their numbers, which costs half of comparing them; what is no GPU (CPU, meta) has -1 in
# common, and is compared as what it is before the call is refused for it.
def _check_rows(what: str, t: torch.Tensor, shape, dtype, cache: PagedCache):
    index = cache.index
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or (index < 0 and t.device != cache.device):
        raise ValueError(f"{what} must be {list(shape)} of {dtype} on {cache.device}, not {list(t.shape)} of {t.dtype} on {t.device}")


def _check_batch(cache: PagedCache, batch: PagedBatch):
    if batch.index != cache.index or (cache.index < 0 and batch.table.device != cache.device):
        raise ValueError("the batch's arrays are on another device than the cache")


def _check_queries(cache: PagedCache, batch: PagedBatch, q: torch.Tensor):
    shape = q.shape
    _check_rows("q", q, (batch.n_rows, shape[1] if len(shape) == 3 else 0, cache.head_dim), cache.row_dtype, cache)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    _check_batch(cache, batch)


# ---------------------------------------------------------------------- calls

def paged_attn_workspace_size(batch: PagedBatch, cfg: AttnConfig) -> int:
    """Bytes of scratch, on the batch's device (they follow its number of SMs)."""
    def size():
        return int(lib().qsa_paged_attn_workspace_size(batch.byref, ctypes.byref(cfg)))
    if not batch.table.is_cuda or batch.table.device.index == torch.cuda.current_device():
        return size()
    with torch.cuda.device(batch.table.device):
        return size()


#: What a configuration says of the tensors of its call.
_CALL_FIELDS = ("n_q_heads", "n_kv_heads", "head_dim", "q_dtype", "kv_dtype", "out_dtype")


def paged_attn(cache: PagedCache, batch: PagedBatch, q: torch.Tensor, out: torch.Tensor,
               lse: torch.Tensor | None = None, *, window: int = 0, n_sinks: int = 0, scale: float = 0.0,
               n_splits: int = 0, workspace: torch.Tensor | None = None, stream=None, cfg: AttnConfig | None = None):
    """Attention of the batch's rows q [n_rows, Hq, D] over their paged caches:
    every token up to the row's own, or with window >= 1 the last `window` of
    them and the first n_sinks tokens."""
    _check_queries(cache, batch, q)
    shape = q.shape
    _check_rows("out", out, shape, out.dtype, cache)
    if lse is not None:
        _check_rows("lse", lse, shape[:2], torch.float32, cache)
    if not (out.is_contiguous() and (lse is None or lse.is_contiguous())):
        raise ValueError("out and lse must be contiguous")
    own = cache._call_config(shape[1], out.dtype, scale, n_splits)
    if cfg is None:
        cfg = own
    elif any(getattr(cfg, f) != getattr(own, f) for f in _CALL_FIELDS):
        raise ValueError("cfg describes another call than the tensors: " + ", ".join(
            f"{f}={getattr(cfg, f)} for {getattr(own, f)}" for f in _CALL_FIELDS if getattr(cfg, f) != getattr(own, f)))
    if workspace is None:
        workspace = _scratch(paged_attn_workspace_size(batch, cfg), cache.device, stream)
    elif workspace.get_device() != cache.index or (cache.index < 0 and workspace.device != cache.device) or (
            not workspace.is_contiguous() or workspace.dtype != torch.uint8):
        raise ValueError(f"workspace must be contiguous uint8 on {cache.device}")
    _call_at("qsa_paged_attn", cache.index, stream, cache.byref, batch.byref, ctypes.byref(cfg), int(window),
          int(n_sinks), q.data_ptr(), out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel())


def paged_append(cache: PagedCache, batch: PagedBatch, k_new: torch.Tensor, v_new: torch.Tensor, stream=None, *,
                 rope: Rope | None = None, q: torch.Tensor | None = None, q_out: torch.Tensor | None = None):
    """Write the batch's rows k_new, v_new ([n_rows, Hkv, D], unit channel stride,
    equal strides: slices of one projection will do) into their pages.  With rope, K
    is rotated for the rows' positions on the way, and q [n_rows, Hq, D] (unit channel
    stride; a slice of the projection will do) into q_out, contiguous, beside it."""
    shape = (batch.n_rows, cache.n_kv_heads, cache.head_dim)
    _check_rows("k_new", k_new, shape, cache.row_dtype, cache)
    _check_rows("v_new", v_new, shape, cache.row_dtype, cache)
    strides = k_new.stride()
    if strides != v_new.stride() or strides[2] != 1:
        raise ValueError("k_new and v_new need unit channel stride and equal strides")
    _check_batch(cache, batch)
    if rope is None:
        if q is not None or q_out is not None:
            raise ValueError("q and q_out go with a rope")
        _call_at("qsa_paged_append", cache.index, stream, cache.byref, batch.byref, cache._row_cfg_ref, k_new.data_ptr(),
              v_new.data_ptr(), strides[0], strides[1])
        return
    cfg, at_q, to_q, q_strides = cache._row_cfg_ref, None, None, (0, 0)
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        q_shape, q_st = q.shape, q.stride()
        if len(q_shape) != 3 or q_st[2] != 1:
            raise ValueError("q must be [n_rows, Hq, D] with unit channel stride")
        _check_rows("q", q, (batch.n_rows, q_shape[1], cache.head_dim), cache.row_dtype, cache)
        _check_rows("q_out", q_out, q_shape, cache.row_dtype, cache)
        if not q_out.is_contiguous():
            raise ValueError("q_out must be contiguous")
        cfg = cache._rows_cfgs.get(q_shape[1]) or cache._rows_cfg(q_shape[1])
        at_q, to_q, q_strides = q.data_ptr(), q_out.data_ptr(), _strides(q_shape, q_st)
    row_stride, head_stride = _strides(shape, strides)
    _call_at("qsa_paged_append_rotate", cache.index, stream, cache.byref, batch.byref, cfg, rope.byref, k_new.data_ptr(),
          v_new.data_ptr(), row_stride, head_stride, at_q, *q_strides, to_q)


def paged_read(cache: PagedCache, batch: PagedBatch, k_out: torch.Tensor, v_out: torch.Tensor, stream=None):
    """The batch's rows back out of their pages, into k_out and v_out ([n_rows, Hkv, D],
    contiguous, both f32 or both bf16); rows without a page are left as they were."""
    shape = (batch.n_rows, cache.n_kv_heads, cache.head_dim)
    if k_out.dtype is not torch.float32 and k_out.dtype is not torch.bfloat16:
        raise TypeError(f"k_out must be float32 or bfloat16, not {k_out.dtype}")
    _check_rows("k_out", k_out, shape, k_out.dtype, cache)
    _check_rows("v_out", v_out, shape, k_out.dtype, cache)
    if not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError("k_out and v_out must be contiguous")
    _check_batch(cache, batch)
    _call_at("qsa_paged_read", cache.index, stream, cache.byref, batch.byref,
          cache._read_cfg[k_out.dtype is torch.bfloat16], k_out.data_ptr(), v_out.data_ptr())


class PagedStep:
    """Preallocated buffers for one layer's attention over its paged cache, so
    the same call can be replayed (or captured in a CUDA graph): `out`, `lse`
    and the workspace belong to the step, and what the table, the lengths and
    the row ranges hold is read when the work runs.

    The buffers are allocated on the stream that is the current one when the step
    is made.  Before its first run on another stream, have that one wait for it
    (Stream.wait_stream): their memory may still be in use by work queued there.
    One step's runs must not overlap each other.

    With a rope, q holds the queries before their rotation (a slice of the projection
    that the new rows are slices of will do), append rotates K and them, these into
    the step's q_rotated, and attend takes that; run then needs the new rows, and attend
    an append before it."""

    def __init__(self, cache: PagedCache, batch: PagedBatch, q: torch.Tensor, *, out_dtype=torch.float32,
                 window: int = 0, n_sinks: int = 0, scale: float = 0.0, n_splits: int = 0, rope: Rope | None = None):
        dev = cache.device
        self.cache, self.batch, self.rope, self.q_in = cache, batch, rope, q
        if rope is not None:
            if q.dim() != 3 or q.stride(2) != 1:
                raise ValueError("q must be [n_rows, Hq, D] with unit channel stride")
            q = self.q_rotated = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _check_queries(cache, batch, q)
        self.q = q
        self._has_q = rope is None
        self.window, self.n_sinks = int(window), int(n_sinks)
        self.cfg = cache.config(q.shape[1], out_dtype, scale, n_splits)
        self.out = torch.empty(q.shape, dtype=out_dtype, device=dev)
        self.lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev)
        self.ws = torch.empty(max(paged_attn_workspace_size(batch, self.cfg), 16), dtype=torch.uint8, device=dev)
        self._args = (cache.byref, batch.byref, ctypes.byref(self.cfg), self.window, self.n_sinks, q.data_ptr(),
                      self.out.data_ptr(), self.lse.data_ptr(), self.ws.data_ptr(), self.ws.numel())

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
        if self.rope is None:
            paged_append(self.cache, self.batch, k_new, v_new, stream)
        else:
            paged_append(self.cache, self.batch, k_new, v_new, stream, rope=self.rope, q=self.q_in, q_out=self.q_rotated)
            self._has_q = True

    def attend(self, stream=None):
        if not self._has_q:
            raise ValueError("a step with a rope attends with the queries that append rotates: append first")
        _call_at("qsa_paged_attn", self.cache.index, stream, *self._args)
        return self.out, self.lse

    def run(self, k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None, stream=None):
        """Append (when given new rows), then attend."""
        if k_new is None and self.rope is not None:
            raise ValueError("a step with a rope rotates q as it appends: give run the new rows (or, after an append, call attend)")
        if k_new is not None:
            self.append(k_new, v_new, stream)
        return self.attend(stream)


@dataclasses.dataclass
class _Caches:
    array: ctypes.Array
    n: int
    cfg: AttnConfig


def _cache_array(caches: Sequence[PagedCache]) -> _Caches:
    caches = list(caches)
    if len({(c.n_kv_heads, c.head_dim, c.kv_dtype, c.page_tokens) for c in caches}) > 1:
        raise ValueError("the caches of a pool have one head layout, dtype and page size")
    arr = (PagedCacheDesc * max(len(caches), 1))(*[c.desc for c in caches])
    return _Caches(arr, len(caches), caches[0].config() if caches else AttnConfig(1, 1, 128, F32, F32, F32, 0.0, 0))


class PagePool:
    """Who holds which page, on the GPU: table [places, pages] (-1: none), lens
    [places] and refs [n_pages] are int32 tensors, and caches are the layers
    whose pages move together.  Every call is asynchronous; requests that could
    not be served are counted (check_device_status) and change nothing.

    step_lens [places] are the lengths for the step that follows an extend, the
    lens of its PagedBatch: those of the pool, and 0 for a place that did not get
    its room, whose rows are then written nowhere and see nothing.  (With the
    pool's own lens such rows would be written over its last tokens.)

    The pool's calls follow each other on one stream, or on streams that the
    caller orders; so does the first of them behind the stream that was the
    current one when the pool was made, where its buffers were allocated."""

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, caches: Sequence[PagedCache] = (),
                 page_tokens: int | None = None):
        if table.dtype != torch.int32 or table.dim() != 2 or not table.is_contiguous():
            raise TypeError("table must be a contiguous int32 [places, pages]")
        _int_list("lens", lens, table)
        _int_list("refs", refs, table)
        if lens.numel() != table.shape[0]:
            raise ValueError("lens must have one entry for each row of table")
        if page_tokens is None:
            if not caches:
                raise ValueError("page_tokens is needed without caches")
            page_tokens = caches[0].page_tokens
        if any(c.device != table.device for c in caches):
            raise ValueError("the pool's arrays are on another device than a cache")
        self.table, self.lens, self.refs, self.caches = table, lens, refs, list(caches)
        self.page_tokens = int(page_tokens)
        self.step_lens = lens.clone()
        self._c = _cache_array(self.caches)
        self.desc = PagePoolDesc(table.data_ptr(), int(table.shape[1]), lens.data_ptr(), refs.data_ptr(),
                                 int(table.shape[0]), int(refs.numel()), self.page_tokens)
        self.byref = ctypes.byref(self.desc)
        self.ws = torch.empty(max(int(lib().qsa_pages_workspace_size(self.byref)), 16), dtype=torch.uint8,
                              device=table.device)
        self._cfg_ref = ctypes.byref(self._c.cfg)

    @classmethod
    def empty(cls, n_places: int, pages_each: int, caches: Sequence[PagedCache]) -> "PagePool":
        """A pool over the caches' pages in which every page is free."""
        dev, n = caches[0].device, min(c.n_pages for c in caches)
        return cls(torch.full((n_places, pages_each), -1, dtype=torch.int32, device=dev),
                   torch.zeros(n_places, dtype=torch.int32, device=dev),
                   torch.zeros(n, dtype=torch.int32, device=dev), caches)

    def _pair(self, a_name, a, b_name, b):
        _int_list(a_name, a, self.table)
        if b is not None and _int_list(b_name, b, self.table).numel() != a.numel():
            raise ValueError(f"{a_name} and {b_name} must have the same length")
        return a.numel()

    def extend(self, seqs: torch.Tensor, n_new: torch.Tensor, stream=None):
        """lens[seqs] += n_new, with the lowest free pages for what they lack; step_lens
        become the lengths of the step."""
        n = self._pair("seqs", seqs, "n_new", n_new)
        _call("qsa_pages_extend_step", self.table.device, stream, self.byref, seqs.data_ptr(), n_new.data_ptr(), n,
              self.step_lens.data_ptr())

    def fork(self, src: torch.Tensor, dst: torch.Tensor, keep: torch.Tensor | None = None, stream=None):
        """The empty places dst become copies of src (their first keep tokens):
        full pages shared, a last page that is not full copied in every cache."""
        n = self._pair("src", src, "dst", dst)
        self._pair("src", src, "keep", keep)
        _call("qsa_pages_fork", self.table.device, stream, self.byref, self._c.array, self._c.n, self._cfg_ref,
                   src.data_ptr(), dst.data_ptr(), _ptr(keep), n, self.ws.data_ptr(), self.ws.numel())

    def free(self, seqs: torch.Tensor, keep: torch.Tensor | None = None, stream=None):
        """Give up the pages of seqs behind their first keep tokens (default: all)."""
        n = self._pair("seqs", seqs, "keep", keep)
        _call("qsa_pages_free", self.table.device, stream, self.byref, seqs.data_ptr(), _ptr(keep), n)

    def compact(self, n_used: torch.Tensor | None = None, stream=None):
        """Move the pages in use to the lowest numbers; n_used (int32, one element
        on the GPU) receives how many there are."""
        if n_used is not None:
            _int_list("n_used", n_used, self.table)
        _call("qsa_pages_compact", self.table.device, stream, self.byref, self._c.array, self._c.n, self._cfg_ref,
                   _ptr(n_used), self.ws.data_ptr(), self.ws.numel())

    def copy(self, src: torch.Tensor, dst: torch.Tensor, stream=None):
        """Copy pages src[i] to dst[i], whole, in every cache."""
        n = self._pair("src", src, "dst", dst)
        _call("qsa_pages_copy", self.table.device, stream, self._c.array, self._c.n, self._cfg_ref, src.data_ptr(),
                   dst.data_ptr(), n)
