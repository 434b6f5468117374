"""Paged attention of values at the ends of their types: NaN as a GPU writes it,
the largest f32 values, fp8 scales of any sign, and queries with a channel far
above the others.  Tolerances are derived in paged_cases."""
import dataclasses

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import Paged, assert_attended, attend64, dev, make_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    qsa.check_device_status()


def run(x: Paged, **kw):
    cache, batch, q = x.device()
    out, lse = torch.empty(q.shape, device=dev()), torch.empty(q.shape[:2], device=dev())
    qsa.paged_attn(cache, batch, q, out, lse, **kw)
    torch.cuda.synchronize()
    assert qsa.check_device_status() == (0, "")
    return out.cpu(), lse.cpu()


# ------------------------------------------------------------------ NaN
#: Bit patterns of NaN: what f32 arithmetic on the GPU returns, its negative, and the smallest and the usual payload.
PATTERNS = {"f32": [0x7FFFFFFF, 0xFFFFFFFF, 0x7F800001, 0xFF800001, 0x7FC00000],
            "bf16": [0x7FFF, 0xFFFF, 0x7F81, 0x7FC0], "fp8": [0x7F, 0xFF]}
NANS = [(d, p) for d, ps in PATTERNS.items() for p in ps]


def set_bits(t: torch.Tensor, at, pattern: int):
    bits = t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])
    width = 8 * t.element_size()
    bits[at] = pattern - (1 << width) if bits.dtype != torch.uint8 and pattern >> (width - 1) else pattern


def nan_case(dtype):
    # A chunk whose rows see different tokens, and a sequence of many key tiles that is split over runs.
    return make_paged([300, 5000], [40, 2], dtype=dtype, D=128, page=32, seed=61)


def place(x: Paged, i: int, t: int):
    return int(x.table[i, t // x.page]), t % x.page


def same_but(good, bad, wrong):
    """Rows (and channels) outside `wrong` hold the same bits, those inside are NaN."""
    assert torch.isnan(bad[wrong]).all()
    assert torch.equal(good[~wrong], bad[~wrong])


@pytest.mark.parametrize("dtype,pattern", NANS + [("fp8", 0x7FFF)])
def test_nan_in_a_query(dtype, pattern):
    if dtype == "fp8" and pattern < 0x100:
        pattern = 0xFF80 | pattern                        # queries of an fp8 cache are bf16
    x = nan_case(dtype)
    good = run(x)
    wrong = torch.zeros(x.q.shape[:2], dtype=torch.bool)
    for r, h in ((3, 1), (39, 23), (41, 7)):
        set_bits(x.q, (r, h, 77), pattern)
        wrong[r, h] = True
    bad = run(x)
    same_but(good[0], bad[0], wrong[..., None].expand_as(bad[0]))
    same_but(good[1], bad[1], wrong)


@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4)])
@pytest.mark.parametrize("dtype,pattern", NANS)
def test_nan_in_a_key(dtype, pattern, window, sinks):
    x = nan_case(dtype)
    good = run(x, window=window, n_sinks=sinks)
    wrong = torch.zeros(x.q.shape[:2], dtype=torch.bool)
    for i, t, h in ((0, 275, 0), (1, 4990, 1), (1, 2, 0)):
        p, s = place(x, i, t)
        set_bits(x.k, (p, h, s, 9), pattern)
        for j in range(x.rows[i]):
            pos = x.lens[i] - x.rows[i] + j
            if t <= pos and (not window or t > pos - window or t < sinks):
                wrong[int(x.row_start[i]) + j, 12 * h:12 * h + 12] = True
    bad = run(x, window=window, n_sinks=sinks)
    assert wrong.any() and not wrong.all()
    same_but(good[0], bad[0], wrong[..., None].expand_as(bad[0]))
    same_but(good[1], bad[1], wrong)


@pytest.mark.parametrize("dtype,pattern", NANS)
def test_nan_in_a_value(dtype, pattern):
    # (Of tokens that every row of their sequence sees: the others' weights are zero, and 0 x NaN is NaN.)
    x = nan_case(dtype)
    good = run(x)
    wrong = torch.zeros(x.q.shape, dtype=torch.bool)
    for i, t, h, c in ((0, 100, 0, 5), (1, 3000, 1, 127)):
        p, s = place(x, i, t)
        set_bits(x.v, (p, h, s, c), pattern)
        wrong[int(x.row_start[i]):int(x.row_start[i + 1]), 12 * h:12 * h + 12, c] = True
    bad = run(x)
    same_but(good[0], bad[0], wrong)
    assert torch.equal(good[1], bad[1])


# ------------------------------------------------------------------ f32
@pytest.mark.parametrize("bits", [0x7F7FFFFF, 0x7F7FF800, 0x7F7FEFFF, 0xFF7FFFFF, 0x7F000000])
def test_f32_values_up_to_the_largest(bits):
    # A row that sees one token returns its V, whose two tf32 parts hold 22 bits: cut off after them, 2^-21 at most.
    x = make_paged([40], [1], dtype="f32", D=128, seed=62)
    p, s = place(x, 0, 39)
    set_bits(x.v, (p, 1, s, 3), bits)
    value = float(x.v[p, 1, s, 3])
    out, lse = run(x, window=1)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert ((out[0, 12:, 3].double() - value).abs() <= 2.0 ** -21 * abs(value)).all()
    # A key of that size against a query that brings the product back to the usual range.
    x = make_paged([40], [1], dtype="f32", D=128, seed=63)
    set_bits(x.k, (p, 1, s, 3), bits)
    x.q[0, :, 3] = 2.0 ** -125
    out, lse = run(x)
    assert_attended(out, lse, attend64(x))


def test_f32_infinities_of_values():
    # The weights' sum over a V with an infinity is that infinity.
    x = make_paged([300, 33], [1, 1], dtype="f32", D=128, seed=64)
    good = run(x)
    p, s = place(x, 0, 120)
    x.v[p, 0, s, 8], x.v[p, 1, s, 9] = float("inf"), float("-inf")
    out, lse = run(x)
    assert (out[0, :12, 8] == float("inf")).all() and (out[0, 12:, 9] == float("-inf")).all()
    out[0, :12, 8], out[0, 12:, 9] = good[0][0, :12, 8], good[0][0, 12:, 9]
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


# ------------------------------------------------------------------ fp8
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 6)])
def test_fp8_scales_of_either_sign_and_zero(D, window, sinks):
    x = make_paged([700, 150, 3], [5, 40, 1], dtype="fp8", D=D, page=32, seed=65, poison=True)
    g = torch.Generator().manual_seed(66)
    pick = torch.rand(x.scale.shape, generator=g)
    x.scale[pick < 0.2] *= -1
    x.scale[pick > 0.9] = 0
    out, lse = run(x, window=window, n_sinks=sinks)
    assert_attended(out, lse, attend64(x, window, sinks))


@pytest.mark.parametrize("bits", [0x7E00, 0xFE00, 0x7FFF, 0xFFFF])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4)])
def test_fp8_scale_of_a_key_that_is_no_number(bits, window, sinks):
    x = nan_case("fp8")
    good = run(x, window=window, n_sinks=sinks)
    wrong = torch.zeros(x.q.shape[:2], dtype=torch.bool)
    for i, t, h in ((0, 275, 0), (1, 4990, 1), (1, 2, 0)):
        p, s = place(x, i, t)
        set_bits(x.scale, (p, h, s, 0), bits)
        for j in range(x.rows[i]):
            pos = x.lens[i] - x.rows[i] + j
            if t <= pos and (not window or t > pos - window or t < sinks):
                wrong[int(x.row_start[i]) + j, 12 * h:12 * h + 12] = True
    bad = run(x, window=window, n_sinks=sinks)
    assert wrong.any() and not wrong.all()
    same_but(good[0], bad[0], wrong[..., None].expand_as(bad[0]))
    same_but(good[1], bad[1], wrong)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("times", [150, 1000, 4000])
def test_fp8_queries_with_a_channel_far_above_the_others(D, times):
    # The keys of that channel are smaller by as much, so that all channels matter to the logits.
    x = make_paged([900, 130], [4, 2], dtype="fp8", D=D, page=32, seed=67)
    x.q[:, :, 5] = x.q[:, :, 5] * times
    x.k[:, :, :, 5] = (torch.randn(x.k.shape[:3], generator=torch.Generator().manual_seed(68)) * 150 / times).to(
        torch.float8_e4m3fn).view(torch.uint8)
    k, v = (c.view(torch.float8_e4m3fn).double() * x.scale[..., w:w + 1].double() for c, w in ((x.k, 0), (x.v, 1)))
    plain = dataclasses.replace(x, k=k, v=v, scale=None)
    ref, l, ref_tol, l_tol = attend64(plain)       # (the bounds of queries that are not split)
    wabs = attend64(dataclasses.replace(plain, v=v.abs()))[0]
    # Q is the sum of two codes, exact from 2^-13 of its row's largest value qmax on and off by dq <= 2^-21 qmax
    # below: logits by up to max_t scale * sum_d dq_d |k_td|, weights by twice that (weight and maximum).
    qmax = x.q.double().abs().amax(-1, keepdim=True)
    dq = torch.where(x.q.double().abs() < 2.0 ** -13 * qmax, torch.minimum(x.q.double().abs(), 2.0 ** -21 * qmax), 0.0)
    for i, n in enumerate(x.lens):
        rows, K = slice(int(x.row_start[i]), int(x.row_start[i + 1])), plain.seq_kv(i)[0]
        lost = torch.einsum("rhgd,htd->rhgt", dq[rows].view(-1, 2, 12, D), K.abs()).amax(-1).flatten(1) * D ** -0.5
        l_tol[rows] += 2 * lost
        ref_tol[rows] += 4 * lost[..., None] * wabs[rows]
    out, lse = run(x)
    assert_attended(out, lse, (ref, l, ref_tol, l_tol))


# ------------------------------------------------------------------ rows to quantize
@pytest.mark.parametrize("D", [128, 256])
def test_fp8_rows_with_nan_keep_it(D):
    # NaN among ordinary values, a row of nothing else, one of NaN and zeros and one of NaN and values whose scale
    # rounds to 0: the codes of NaN are NaN, the others as without it.
    n = 6
    g = torch.Generator().manual_seed(69)
    k_new, v_new = (torch.randn(n, 2, D, generator=g).bfloat16() for _ in range(2))
    k_new[1, 0, 7] = k_new[1, 1, D - 1] = float("nan")
    v_new[2] = float("nan")
    k_new[3] = 0
    k_new[3, 0, ::3] = float("nan")
    v_new[4] = 1e-9
    v_new[4, 1, 5] = float("nan")
    set_bits(k_new, (5, 0, 0), 0xFFFF)
    rows = [t.clone() for t in (k_new, v_new)]
    for t in rows:
        t[torch.isnan(t)] = 0
    caches, state = [], []
    one = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev())
    for k, v in (rows, (k_new, v_new)):
        cache = qsa.PagedCache(*(torch.zeros(1, 2, 16, D, dtype=torch.uint8, device=dev()) for _ in range(2)),
                               torch.zeros(1, 2, 16, 2, dtype=torch.float16, device=dev()))
        qsa.paged_append(cache, qsa.PagedBatch(one(0)[None], one(n), one(0, n), n_rows=n), k.to(dev()), v.to(dev()))
        caches.append(cache)
        state.append([cache.k[0, :, :n].cpu(), cache.v[0, :, :n].cpu(), cache.kv_scale.cpu()])
    for was, now, x in zip(state[0], state[1], (k_new, v_new)):
        nan = torch.isnan(x).transpose(0, 1)
        assert ((now & 0x7F) == 0x7F)[nan].all() and torch.equal(now[~nan], was[~nan])
    assert torch.equal(state[0][2], state[1][2])
    # The append into segments gives the same codes ...
    seg = [torch.zeros(2, 16, D, dtype=torch.uint8, device=dev()) for _ in range(2)]
    sc = torch.zeros(2, 16, 2, dtype=torch.float16, device=dev())
    seq = qsa.Seq(n, n, torch.zeros(4, 128, device=dev()), [qsa.Segment(seg[0], seg[1], 0, sc)],
                  idx_keys=torch.zeros(16, 128, dtype=torch.bfloat16, device=dev()))
    qsa.append_tokens(seq, k_new.transpose(0, 1).contiguous().to(dev()), v_new.transpose(0, 1).contiguous().to(dev()),
                      torch.zeros(n, 128, dtype=torch.bfloat16, device=dev()))
    assert torch.equal(caches[1].k[0], seg[0]) and torch.equal(caches[1].v[0], seg[1])
    assert torch.equal(caches[1].kv_scale[0], sc)
    # ... and rows that see such a token are NaN.
    q = torch.randn(n, 4, D, generator=g).bfloat16().to(dev())
    out, lse = torch.empty(q.shape, device=dev()), torch.empty(q.shape[:2], device=dev())
    qsa.paged_attn(caches[1], qsa.PagedBatch(one(0)[None], one(n), one(0, n), n_rows=n), q, out, lse, window=1)
    nan_k, nan_v = torch.isnan(k_new).any(-1), torch.isnan(v_new)
    assert torch.equal(torch.isnan(lse.cpu()), nan_k.repeat_interleave(2, 1))
    for r in (2, 5):                                      # (rows of one token, the others' weights are zero)
        last = qsa.PagedBatch(one(0)[None], one(r + 1), one(0, 1), n_rows=1)
        qsa.paged_attn(caches[1], last, q[r:r + 1], out[r:r + 1], lse[r:r + 1], window=1)
        want = (nan_k[r][:, None] | nan_v[r]).repeat_interleave(2, 0)
        assert torch.equal(torch.isnan(out[r].cpu()), want)
