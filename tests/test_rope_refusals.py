"""Rotations and 4-bit paged caches without a GPU: frequencies, refusals, and the
plain 4-bit codec of the tests (device pointers are fake aligned addresses)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from indexed_sparse_attention_gb300 import build as qsa_build
from indexed_sparse_attention_gb300 import paged, rope
from q4_cases import encode4, order4, split4

FAKE, MIS = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    qsa_build.build()
    return qsa.lib()


def _rope(L, **kw):
    r = qsa.Rope(64).desc
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_frequencies(L):
    w = qsa.Rope(128, base=1e6).frequencies
    assert len(w) == 64 and all(math.isclose(a, 1e6 ** (-2 * i / 128), rel_tol=1e-14) for i, a in enumerate(w))
    lin = qsa.Rope(128, base=1e6, scaling=qsa.RopeScaling("linear", 8.0))
    assert all(math.isclose(a, b / 8, rel_tol=1e-15) for a, b in zip(lin.frequencies, w)) and lin.magnitude == 1.0
    parts = qsa.Rope(128, base=1e6, scaling=qsa.RopeScaling("parts", 32.0, original_tokens=8192, fast=32, slow=1))
    turns = [8192 * a / (2 * math.pi) for a in w]
    assert turns[0] > 32 and turns[-1] < 1 and any(1 < t < 32 for t in turns)
    for a, b, t in zip(parts.frequencies, w, turns):
        if t >= 32:
            assert a == b
        elif t <= 1:
            assert math.isclose(a, b / 32, rel_tol=1e-15)
        else:
            assert b / 32 < a < b
    assert math.isclose(parts.magnitude, 0.1 * math.log(32) + 1, rel_tol=1e-6)
    assert qsa.Rope(32, frequencies=[0.5] * 16, magnitude=2.0).magnitude == 2.0
    assert qsa.Rope(128, scaling=qsa.RopeScaling("parts", 1.0, original_tokens=100)).magnitude == 1.0


def test_angles_are_64_bit_turns(L):
    for w in (1.0, 0.3, 1e-6, 3.14159, -0.7, 0.0, 7.5):
        t = qsa.Rope(16, frequencies=[w] * 8).desc.turns[0]
        exact = Fraction(w) / (2 * Fraction(math.pi))     # (pi to binary64: 2^-53 of it)
        off = (Fraction(t, 1 << 64) - exact) % 1
        off = min(off, 1 - off)
        assert off <= abs(exact) * Fraction(1, 1 << 51) + Fraction(1, 1 << 60)


def test_rope_checks(L):
    w, mag = (ctypes.c_double * 128)(*[0.1] * 128), ctypes.c_float()
    f = lambda d=64, base=1e4, kind=0, factor=1.0, n=0.0, fast=32.0, slow=1.0, to=w, m=ctypes.byref(mag): \
        L.qsa_rope_frequencies(d, base, kind, factor, n, fast, slow, to, m)
    assert f() == 0 and f(to=None) == 1 and f(m=None) == 1
    assert f(d=0) == 2 and f(d=24) == 2 and f(d=272) == 2 and f(d=-16) == 2 and f(kind=3) == 2 and f(kind=-1) == 2
    assert f(base=0.5) == 1 and f(base=math.nan) == 1 and f(base=math.inf) == 1
    assert f(kind=1, factor=0.5) == 1 and f(kind=1, factor=math.nan) == 1 and f(kind=0, factor=math.nan) == 0
    assert f(kind=2, factor=2.0) == 1 and f(kind=2, factor=2.0, n=100.0, fast=1.0) == 1
    assert f(kind=2, factor=2.0, n=100.0, slow=-1.0) == 1 and f(kind=2, factor=2.0, n=100.0) == 0
    r = rope.RopeDesc()
    init = lambda d=64, pairs=0, to=w, m=1.0, out=r: L.qsa_rope_init(out, d, pairs, to, m)
    assert init() == 0 and init(out=None) == 1 and init(to=None) == 1 and init(d=20) == 2 and init(d=512) == 2
    assert init(pairs=2) == 1 and init(m=math.inf) == 1
    w[3] = math.nan
    assert init() == 1 and "frequency 3" in L.qsa_last_error().decode()


def test_rotate_checks(L):
    r = _rope(L)
    call = lambda rope=r, pos=FAKE, rows=4, heads=2, dim=128, kind=1, x=FAKE, xr=256, xh=128, y=FAKE * 2, yr=256, yh=128: \
        L.qsa_rotate(rope, pos, rows, heads, dim, kind, x, xr, xh, y, yr, yh, None)
    assert call(rope=None) == 1 and call(pos=None) == 1 and call(x=None) == 1 and call(y=None) == 1
    assert call(rows=-1) == 1 and call(heads=-1) == 1 and call(heads=1 << 17) == 2
    assert call(dim=100) == 2 and call(dim=0) == 2 and call(dim=2048) == 2 and call(dim=48) == 1
    assert call(kind=2) == 2 and call(kind=4) == 2 and call(kind=-1) == 2
    assert call(x=MIS) == 3 and call(y=MIS) == 3 and call(xr=260) == 3 and call(xh=132) == 3 and call(yr=512, yh=132) == 3 and call(pos=FAKE + 2) == 3
    assert call(xr=-256) == 1 and call(yr=64) == 1 and call(yh=0) == 1 and call(xr=1 << 41) == 1
    assert call(yr=128, yh=128) == 1                       # rows over heads
    assert call(y=FAKE, yr=512) == 1                       # in place with other strides
    for bad in (_rope(L, rot_dim=24), _rope(L, rot_dim=0), _rope(L, rot_dim=1 << 20)):
        assert call(rope=bad) == 2
    assert call(rope=_rope(L, pairs=3)) == 1 and call(rope=_rope(L, magnitude=math.nan)) == 1
    assert call(rows=0, x=None, y=None, pos=None) == 0 and call(heads=0, x=None) == 0


def _cache(**kw):
    c = paged.PagedCacheDesc(FAKE, FAKE, 2 * 16 * 128, 16 * 128, 128, FAKE, 32, 16, 1, 10, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(**kw):
    b = paged.PagedBatchDesc(FAKE, 8, FAKE, FAKE, 2, 3, 2)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _cfg(**kw):
    c = qsa.AttnConfig(24, 2, 128, qsa.BF16, qsa.Q4, qsa.F32, 0.0, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("want,cache,cfg", [
    (1, {"kv_scale": None}, {}), (3, {"kv_scale": 0x10008}, {}), (1, {"scale_tok_stride": 0}, {}),
    (1, {"scale_head_stride": -1}, {}), (1, {"scale_page_stride": 1 << 40}, {}), (3, {"tok_stride": 144}, {}),
    (3, {"head_stride": 2049}, {}), (3, {"page_stride": 4112}, {}), (1, {"tok_stride": 64}, {}), (3, {"k": MIS}, {}),
    (2, {"page_tokens": 24}, {}), (2, {}, {"q_dtype": qsa.F32}), (2, {}, {"head_dim": 64}), (2, {}, {"out_dtype": qsa.Q4}),
    (2, {}, {"kv_dtype": 5}), (2, {}, {"kv_dtype": -1}), (2, {}, {"q_dtype": qsa.Q4})])
def test_q4_cache_checks(L, want, cache, cfg):
    c, b, g = _cache(**cache), _batch(), _cfg(**cfg)
    assert L.qsa_paged_attn(c, b, g, 0, 0, FAKE, FAKE, None, FAKE, 1 << 40, None) == want
    assert L.qsa_paged_append(c, b, g, FAKE, FAKE, 256, 128, None) == want
    assert L.qsa_paged_append_rotate(c, b, g, _rope(L), FAKE, FAKE, 256, 128, FAKE, 24 * 128, 128, FAKE, None) == want
    assert L.qsa_paged_read(c, b, g, FAKE, FAKE, None) == want
    pool = paged.PagePoolDesc(FAKE, 8, FAKE, FAKE, 4, 10, 16)
    assert L.qsa_pages_fork(pool, c, 1, g, FAKE, FAKE, None, 2, FAKE, 1 << 40, None) == want
    assert L.qsa_pages_copy(c, 1, g, FAKE, FAKE, 2, None) == want


def test_4_bits_are_for_paged_caches_only(L):
    seq = (qsa.SeqDesc * 1)()
    seq[0].n_tokens, seq[0].n_rows, seq[0].n_segments = 8, 1, 1
    assert L.qsa_sparse_attn(seq, 1, _cfg(), FAKE, FAKE, FAKE, 512, FAKE, None, FAKE, 1 << 30, None) == 2
    assert L.qsa_attn_workspace_size(seq, 1, _cfg(), 512) == 0
    need = L.qsa_paged_attn_workspace_size(_batch(), _cfg())
    assert need > 0
    assert L.qsa_paged_attn(_cache(), _batch(), _cfg(), 0, 0, FAKE, FAKE, None, FAKE, need - 1, None) == 4


def test_append_rotate_and_read_checks(L):
    r = _rope(L)
    call = lambda rope=r, k=FAKE, v=FAKE, rs=256, hs=128, q=FAKE, qr=24 * 128, qh=128, qo=FAKE * 2, b=_batch(), g=_cfg(): \
        L.qsa_paged_append_rotate(_cache(), b, g, rope, k, v, rs, hs, q, qr, qh, qo, None)
    assert call(rope=None) == 1 and call(k=None) == 1 and call(v=None) == 1 and call(qo=None) == 1
    assert call(k=MIS) == 3 and call(rs=260) == 3 and call(q=MIS) == 3 and call(qo=MIS) == 3 and call(qr=1028) == 3
    assert call(rs=-256) == 1 and call(qh=-128) == 1
    assert call(rope=_rope(L, rot_dim=144)) == 1 and call(rope=_rope(L, rot_dim=8)) == 2
    assert call(qo=FAKE, qr=28 * 128) == 1 and call(qo=FAKE, qh=256) == 1         # in place: contiguous
    assert call(b=_batch(n_rows=0), k=None, qo=None) == 0 and call(b=_batch(table=None)) == 1
    read = lambda k=FAKE, v=FAKE, b=_batch(), g=_cfg(): L.qsa_paged_read(_cache(), b, g, k, v, None)
    assert read(k=None) == 1 and read(v=None) == 1 and read(k=MIS) == 3 and read(v=MIS) == 3
    assert read(b=_batch(n_seqs=0), k=None) == 0 and read(g=_cfg(n_splits=-1)) == 1


def test_python_refusals(L):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    f16 = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache = qsa.PagedCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), f16(4, 2, 16, 16), kv_dtype=qsa.Q4)
    assert cache.head_dim == 128 and cache.desc.tok_stride == 128 and cache.desc.scale_tok_stride == 1
    assert cache.desc.head_stride == 16 * 128 and cache.desc.scale_head_stride == 16 and cache.row_dtype is torch.bfloat16
    with pytest.raises(ValueError):
        qsa.PagedCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), kv_dtype=qsa.Q4)
    with pytest.raises(TypeError, match="kv_scale"):
        qsa.PagedCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), f16(4, 2, 16, 2), kv_dtype=qsa.Q4)
    with pytest.raises(TypeError, match="kv_scale"):
        qsa.PagedCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), f16(4, 2, 16, 24)[..., :16], kv_dtype=qsa.Q4)
    with pytest.raises(TypeError, match="does not hold"):
        qsa.PagedCache(u8(4, 2, 16, 64).bfloat16(), u8(4, 2, 16, 64).bfloat16(), f16(4, 2, 16, 16), kv_dtype=qsa.Q4)
    with pytest.raises(TypeError, match="does not hold"):
        qsa.PagedCache(u8(4, 2, 16, 64), u8(4, 2, 16, 64), f16(4, 2, 16, 2), kv_dtype=qsa.BF16)
    with pytest.raises(ValueError):
        qsa.PagedCache.zeros(4, 2, 16, 128, qsa.Q8, device="cpu")
    for kind in (qsa.F32, qsa.BF16, qsa.FP8, qsa.Q4):
        c = qsa.PagedCache.zeros(4, 2, 16, 256, kind, device="cpu")
        assert c.head_dim == 256 and c.kv_dtype == kind
    batch = qsa.PagedBatch(i32(2, 4), i32(2), i32(3), n_rows=2)
    rows, q = torch.zeros(2, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 24, 128, dtype=torch.bfloat16)
    r = qsa.Rope(64)
    put = lambda **kw: qsa.paged_append(cache, batch, rows, rows, **kw)
    for kw, why in (({"q": q, "q_out": q}, "go with a rope"), ({"rope": r, "q": q}, "go together"),
                    ({"rope": r, "q": q[:1], "q_out": q}, "q must be"), ({"rope": r, "q": q, "q_out": q.float()}, "q_out must be"),
                    ({"rope": r, "q": q, "q_out": torch.zeros(2, 48, 128, dtype=torch.bfloat16)[:, ::2]}, "contiguous"),
                    ({"rope": r, "q": q, "q_out": q.clone()}, "not on a GPU")):
        with pytest.raises(ValueError, match=why):
            put(**kw)
    with pytest.raises(TypeError):
        qsa.paged_read(cache, batch, rows.half(), rows.half())
    with pytest.raises(ValueError, match="v_out must be"):
        qsa.paged_read(cache, batch, rows, rows.float())
    with pytest.raises(ValueError, match="not on a GPU"):
        qsa.paged_read(cache, batch, rows, rows.clone())
    pos = i32(2)
    for bad in ((pos.long(), q), (pos[:1], q), (i32(4)[::2], q)):
        with pytest.raises(TypeError, match="positions"):
            qsa.rotate(r, *bad)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        qsa.rotate(r, pos, q.half())
    with pytest.raises(ValueError):
        qsa.rotate(r, pos, q, q[:, :12])
    with pytest.raises(ValueError, match="unit channel"):
        qsa.rotate(r, pos, q.transpose(1, 2))
    with pytest.raises(ValueError, match="not on a GPU"):
        qsa.rotate(r, pos, q)
    for kw in ({"scaling": qsa.RopeScaling("odd", 2.0)}, {"frequencies": [1.0] * 31},
               {"frequencies": [1.0] * 32, "scaling": qsa.RopeScaling("linear", 2.0)}):
        with pytest.raises(ValueError):
            qsa.Rope(64, **kw)
    for d in (0, 8, 40, 512):
        with pytest.raises(qsa.QSAError):
            qsa.Rope(d)


@pytest.mark.parametrize("D", [128, 256])
def test_the_plain_4_bit_codec(D):
    """The tests' own codec: a round trip is off by at most half a step (and the minimum's rounding)."""
    assert sorted(order4(D).tolist()) == list(range(D)) and order4(D)[:8].tolist() == [0, 1, 2, 3, *(4 * (D // 32) + i for i in range(4))]
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(40, D, generator=g) * torch.logspace(-3, 3, 40)[:, None]).bfloat16().float()
    x[3], x[4] = 0.0, 2.5
    code, s, m = split4(*encode4(x))
    err = (code * s + m - x.double()).abs()
    assert (err <= s * 0.5 + (x.double().abs().amax(-1, keepdim=True) * 2.0 ** -10 + 2.0 ** -24)).all()
    x[5, 7], x[6, 40], x[7, 0] = float("nan"), float("inf"), 1e6
    code, s, m = split4(*encode4(x))
    assert torch.isnan(s[5, :32]).all() and torch.isfinite(s[5, 32:]).all()
    assert torch.isnan(s[6, 32:64]).all() and torch.isnan(s[7, :32]).all()
