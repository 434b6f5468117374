"""Paged K/V caches on the GPU: attention (whole and windowed) against 64 bits,
rows written into pages, the keeping of pages against plain Python, and a run
of them together.  Tolerances are derived in paged_cases."""
import random

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import Paged, Pool, assert_attended, attend64, dev, encode_fp8, make_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    qsa.check_device_status()


def run(x: Paged, *, out_dtype=torch.float32, window=0, sinks=0, n_splits=0, scale=0.0):
    cache, batch, q = x.device()
    out = torch.full(q.shape, 7.0, dtype=out_dtype, device=dev())
    lse = torch.full(q.shape[:2], 7.0, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse, window=window, n_sinks=sinks, n_splits=n_splits, scale=scale)
    torch.cuda.synchronize()
    return out, lse


def check(x, **kw):
    ref = attend64(x, kw.get("window", 0), kw.get("sinks", 0), kw.get("scale") or None)
    out, lse = run(x, **kw)
    assert_attended(out, lse, ref, sum(x.rows))
    assert qsa.check_device_status() == (0, "")
    return out, lse


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("D,page,order", [(128, 16, "head"), (256, 32, "token"), (256, 64, "head"), (128, 256, "token")])
def test_decode_and_verify_ragged(dtype, D, page, order):
    # Lengths of one, around page and tile ends, and long enough to be split.
    x = make_paged([1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700, 2049], [1, 2, 1, 4, 3, 1, 1, 2, 1, 8, 5, 1, 2],
                   dtype=dtype, D=D, page=page, order=order, seed=1, poison=True)
    check(x)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (100, 5), (128, 64), (129, 128), (500, 130),
                                          (1 << 30, 9), (200, 1 << 30)])
def test_windows_and_sinks(dtype, window, sinks):
    x = make_paged([1, 40, 300, 777, 1025], [1, 2, 9, 1, 30], dtype=dtype, D=128, page=32, seed=2, poison=True)
    check(x, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 10)])
def test_chunks_of_rows(dtype, D, window, sinks):
    # Chunks that begin their sequence and that follow a prefix, next to single rows.
    x = make_paged([200, 333, 64, 1], [200, 97, 1, 1], dtype=dtype, D=D, page=16, order="token", seed=3, poison=True)
    check(x, window=window, sinks=sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (8, 1), (3, 5), (1, 16), (4, 8), (2, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_layouts(Hkv, G, dtype):
    x = make_paged([90, 411, 33], [3, 17, 33], dtype=dtype, D=128, Hkv=Hkv, G=G, page=64, seed=4, poison=True)
    check(x)


def test_page_sizes_and_scale():
    for page in (16, 32, 64, 128, 256, 512, 1024):
        x = make_paged([1100, 5, 513], [2, 1, 4], dtype="bf16", D=128, page=page, seed=page, poison=True)
        check(x, scale=0.05)


def test_steps_at_once_on_two_streams():
    # Two steps with their own workspaces, plain and captured, interleaved on two streams.
    cases = [make_paged([3000, 40, 700], [4, 1, 30], dtype=d, D=D, page=32, seed=45) for d, D in (("bf16", 256), ("fp8", 128))]
    steps, alone, graphs = [], [], []
    streams = [torch.cuda.Stream() for _ in cases]
    for x in cases:
        cache, batch, q = x.device()
        steps.append(qsa.PagedStep(cache, batch, q, window=900, n_sinks=5))
    for st in steps:
        out, lse = st.attend()
        torch.cuda.synchronize()
        alone.append((out.clone(), lse.clone()))
    for st, stream in zip(steps, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            for _ in range(3):
                st.attend()
        graphs.append(g)
    for turn in range(10):
        for st, stream, g in zip(steps, streams, graphs):
            with torch.cuda.stream(stream):
                st.out.zero_()
                if turn % 2:
                    g.replay()
                else:
                    for _ in range(4):
                        st.attend()
        torch.cuda.synchronize()
        for st, (out, lse) in zip(steps, alone):
            assert torch.equal(st.out, out) and torch.equal(st.lse, lse)
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("D,page", [(128, 16), (256, 1024)])
def test_caches_that_are_views(dtype, D, page):
    # K and V side by side in one tensor of pages, of which every second one is the cache's; scales likewise.
    x = make_paged([1500, 70, 3], [4, 1, 2], dtype=dtype, D=D, page=page, seed=44, poison=True)
    n, Hkv = x.k.shape[:2]
    kv = torch.zeros(2 * n, 2, Hkv, page, D, dtype=x.k.dtype, device=dev())
    kv[::2, 0], kv[::2, 1] = x.k.to(dev()), x.v.to(dev())
    sc = None
    if x.scale is not None:
        sc = torch.zeros(2 * n, page, Hkv, 2, dtype=torch.float16, device=dev()).transpose(1, 2)
        sc[::2] = x.scale.to(dev())
        sc = sc[::2]
    _, batch, q = x.device()
    cache = qsa.PagedCache(kv[::2, 0], kv[::2, 1], sc)
    out, lse = torch.empty(q.shape, device=dev()), torch.empty(q.shape[:2], device=dev())
    for window, sinks in ((0, 0), (90, 7)):
        qsa.paged_attn(cache, batch, q, out, lse, window=window, n_sinks=sinks)
        torch.cuda.synchronize()
        assert_attended(out, lse, attend64(x, window, sinks))
    before = kv.clone()
    rows = torch.ones(q.shape[0], Hkv, D, dtype=cache.row_dtype, device=dev())
    qsa.paged_append(cache, batch, rows, 2 * rows)
    torch.cuda.synchronize()
    assert torch.equal(kv[1::2].view(torch.uint8), before[1::2].view(torch.uint8))   # the pages between are not the cache's
    assert not torch.equal(kv[::2].view(torch.uint8), before[::2].view(torch.uint8))
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("D", [128, 256])
def test_queries_of_any_size(dtype, D):
    # A channel far above the others, rows of zeros, of the smallest and of large values, next to ordinary ones.
    x = make_paged([400, 130, 5], [9, 1, 2], dtype=dtype, D=D, seed=31, poison=True)
    x.q[0, :, 5] *= 150
    x.q[1] *= 2.0 ** -110
    x.q[2] = 0
    x.q[3] *= 2.0 ** -130
    x.q[4, :, D - 1] = 2.0 ** -120
    x.q[5, 1::2] *= 300
    x.q[9, :, :D // 2] *= 0.001
    check(x)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_queries_that_are_no_numbers_stay_in_their_rows(dtype):
    x = make_paged([300, 40], [5, 2], dtype=dtype, D=128, seed=32)
    good = run(x)
    x.q[1, 3, 7] = float("nan")
    x.q[2, 4, 100] = float("inf")
    bad = run(x)
    rows = torch.ones(x.q.shape[:2], dtype=torch.bool)
    rows[1, 3] = rows[2, 4] = False
    for a, b in zip(good, bad):
        assert torch.equal(a.cpu()[rows], b.cpu()[rows])
    assert torch.isnan(bad[0][1, 3]).all() and torch.isnan(bad[0][2, 4]).all()
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_tokens_outside_the_window_may_hold_anything(dtype):
    # Everything before the window and behind the sinks is NaN: in K, in V and in the scales.
    W, S, n, r = 100, 20, 600, 3
    x = make_paged([n], [r], dtype=dtype, D=256, page=16, seed=5, poison=True)
    for t in range(S, n - r - W + 1):
        p, s = int(x.table[0, t // 16]), t % 16
        if dtype == "fp8":
            x.k[p, :, s], x.v[p, :, s], x.scale[p, :, s] = 0x7F, 0x7F, float("inf")
        else:
            x.k[p, :, s], x.v[p, :, s] = float("nan"), float("-inf")
    check(x, window=W, sinks=S)


def test_rows_that_see_nothing_and_rows_of_nobody():
    # Empty sequences, sequences without rows, more rows than tokens, and rows outside every range.
    x = make_paged([50, 0, 30, 3], [2, 0, 0, 3], dtype="bf16", page=16, seed=6, pad_rows=5)
    cache, batch, q = x.device()
    # Sequence 1 has no tokens but a row, and sequence 3 has 3 tokens and 5 rows; a row before the first range.
    start = torch.tensor([1, 3, 4, 4, 9], dtype=torch.int32, device=dev())
    batch = qsa.PagedBatch(batch.table, batch.lens, start, n_rows=q.shape[0], max_rows=5)
    out = torch.full(q.shape, 7.0, device=dev())
    lse = torch.full(q.shape[:2], 7.0, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse)
    y = Paged(x.k, x.v, None, x.table, [50, 0, 30, 3], [2, 0, 0, 3], torch.tensor([1, 3, 3, 3, 6]), None, 16, "head")
    y.q = torch.cat((x.q[:3], x.q[6:9]))                # (rows 4 and 5 of the batch are at positions -2 and -1)
    y.row_start = torch.tensor([1, 3, 3, 3, 6])
    ref = attend64(y)
    keep = [1, 2, 6, 7, 8]
    assert_attended(out[keep], lse[keep], tuple(t[[1, 2, 3, 4, 5]] for t in ref))
    for r in (3, 4, 5):                                  # nothing visible
        assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    for r in (0, 9):                                     # nobody's rows
        assert (out[r] == 7).all() and (lse[r] == 7).all()
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_divisions_agree_and_repeat(dtype):
    x = make_paged([3000, 70, 900], [4, 1, 2], dtype=dtype, D=128, page=64, seed=7)
    ref = attend64(x)
    for n in (1, 2, 3, 7, 50, 0):
        out, lse = run(x, n_splits=n)
        assert_attended(out, lse, ref)
        for _ in range(5):
            again, lse2 = run(x, n_splits=n)
            assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("D", [128, 256])
def test_one_run_of_short_items(dtype, D):
    # The roles of a run work on different items at once, one to three tiles each.
    lens = [1 + (37 * i) % 390 for i in range(40)]
    x = make_paged(lens, [1 + i % 3 if n > 3 else 1 for i, n in enumerate(lens)], dtype=dtype, D=D, page=32, seed=33)
    for n in (1, 2, 5):
        first = check(x, n_splits=n)
        for _ in range(10):
            again = run(x, n_splits=n)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_outputs_and_workspaces_on_16_bytes(dtype, out_dtype):
    # Addresses that are multiples of 16 but not of 32.
    x = make_paged([700, 9, 40], [4, 1, 40], dtype=dtype, D=128, page=64, seed=14)
    cache, batch, q = x.device()
    cfg = cache.config(24, out_dtype)
    need = qsa.paged_attn_workspace_size(batch, cfg)
    ws = torch.empty(need + 16, dtype=torch.uint8, device=dev())[16:]
    es = torch.empty(0, dtype=out_dtype).element_size()
    out = torch.empty(q.numel() + 16 // es, dtype=out_dtype, device=dev())[16 // es:].view(q.shape)
    q2 = torch.empty(q.numel() + 16 // q.element_size(), dtype=q.dtype, device=dev())[16 // q.element_size():].view(q.shape)
    q2.copy_(q)
    lse = torch.empty(q.numel() // 128 + 1, device=dev())[1:].view(q.shape[:2])
    assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    qsa.paged_attn(cache, batch, q2, out, lse, workspace=ws, cfg=cfg)
    assert_attended(out, lse, attend64(x))


def test_many_sequences():
    # More sequences than a CTA has threads: the division takes its two passes.
    rng = random.Random(8)
    lens = [rng.randint(1, 90) for _ in range(700)]
    rows = [rng.choice([0, 1, 1, 2]) if n > 1 else 1 for n in lens]
    x = make_paged(lens, rows, dtype="bf16", Hkv=1, G=4, page=16, seed=8, poison=True)
    check(x)
    check(x, window=20, sinks=2)


def test_a_long_chunk_next_to_short_ones():
    # A sequence of many items among short ones, before, between and behind.
    x = make_paged([5, 900, 7, 700, 3], [1, 900, 2, 650, 1], dtype="bf16", Hkv=1, G=8, page=32, seed=9, poison=True)
    check(x, out_dtype=torch.bfloat16)
    check(x, window=128, sinks=4, n_splits=5)


def test_pages_past_32_bits():
    # Page offsets above 2^31 elements: page 40,000 of 64 x 2 x 512 elements begins at element 2.6e9.
    page, n_pages = 64, 40_002
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 12 GB")
    x = make_paged([100], [2], dtype="bf16", D=256, page=page, seed=10)
    k = torch.empty(n_pages, 2, page, 512, dtype=torch.bfloat16, device=dev())[..., :256]
    v = torch.empty(n_pages, 2, page, 512, dtype=torch.bfloat16, device=dev())[..., :256]
    at = [40_001, 39_999]
    for j, p in enumerate(at):
        k[p], v[p] = x.k[x.table[0, j]].to(dev()), x.v[x.table[0, j]].to(dev())
    table = torch.tensor([at], dtype=torch.int32, device=dev())
    lens = torch.tensor([100], dtype=torch.int32, device=dev())
    batch = qsa.PagedBatch(table, lens, torch.tensor([0, 2], dtype=torch.int32, device=dev()), n_rows=2)
    cache = qsa.PagedCache(k, v)
    q = x.q.to(dev())
    out, lse = torch.empty(2, 24, 256, device=dev()), torch.empty(2, 24, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse)
    assert_attended(out, lse, attend64(x))
    new = torch.randn(2, 2, 256, device=dev()).bfloat16()
    qsa.paged_append(cache, batch, new, new)
    assert torch.equal(k[39_999, :, 34:36], new.transpose(0, 1)) and torch.equal(v[39_999, :, 34:36], new.transpose(0, 1))
    pool = qsa.PagePool(table, lens, torch.zeros(n_pages, dtype=torch.int32, device=dev()), [cache])
    pool.copy(torch.tensor([40_001], dtype=torch.int32, device=dev()), torch.tensor([39_000], dtype=torch.int32, device=dev()))
    assert torch.equal(k[39_000], k[40_001]) and torch.equal(v[39_000], v[40_001])


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_lengths_and_windows_at_the_ends_of_32_bits(dtype):
    # A length behind every table: only the first tokens have pages, and the window's are skipped.
    x = make_paged([40, 40], [3, 2], dtype=dtype, D=128, seed=41)
    cache, batch, q = x.device()
    out, lse = torch.full(q.shape, 7.0, device=dev()), torch.full(q.shape[:2], 7.0, device=dev())
    batch.lens[0] = 2 ** 31 - 1
    qsa.paged_attn(cache, batch, q, out, lse, window=64, n_sinks=40)
    torch.cuda.synchronize()
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK
    seen = Paged(x.k, x.v, x.scale, x.table, [40], [3], x.row_start[:2], x.q[:3], x.page, x.order)
    K, V = (t.float() for t in seen.seq_kv(0))
    G = x.q.shape[1] // K.shape[0]
    z = torch.einsum("rhgd,htd->rhgt", x.q[:3].float().view(3, -1, G, 128), K) * 128 ** -0.5
    want = torch.einsum("rhgt,htd->rhgd", z.softmax(-1), V).reshape(3, -1, 128)
    # Weights rounded to bf16 (2^-8 of the largest value), the rest in 32 bits.
    assert (out[:3].cpu() - want).abs().max() < ((0 if dtype == "f32" else 2.0 ** -8) + 1e-4) * V.abs().max()
    # Windows longer than any sequence, rows before the first token among the others.
    x = make_paged([3, 50], [3, 2], dtype=dtype, D=128, seed=42)
    a, b = run(x), run(x, window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cache, batch, q = x.device()
    batch.lens[0] = 1                                          # rows at positions -2, -1 and 0
    for window in (0, 2 ** 31 - 1, 2 ** 31 - 2 ** 26):
        qsa.paged_attn(cache, batch, q, out[:5], lse[:5], window=window)
        torch.cuda.synchronize()
        assert (out[:2] == 0).all() and torch.isinf(lse[:2]).all() and torch.isfinite(lse[2:5]).all()
    assert qsa.check_device_status() == (0, "")


def test_windows_whose_items_differ_by_a_tile():
    # Items of 2,731 and 2,730 tiles of 32 tokens by three heads: 8,193 and 8,190.
    Hkv, D, P, W = 3, 128, 1024, 2730 * 32 - 20
    fits = [n for n in range(W + 200, W + 232)
            if (-(-(n - 8) // 32) - (n - 40 - W + 1) // 32, -(-n // 32) - (n - 8 - W + 1) // 32) == (2731, 2730)]
    n = fits[0]
    pages = -(-n // P)
    g = torch.Generator(device="cuda").manual_seed(43)
    k, v = (torch.randn(pages, Hkv, P, D, device=dev(), generator=g) for _ in range(2))
    q = torch.randn(40, Hkv, D, device=dev(), generator=g)
    table = torch.arange(pages, dtype=torch.int32, device=dev())[None].contiguous()
    batch = qsa.PagedBatch(table, _ints([n]), _ints([0, 40]), n_rows=40)
    out, lse = torch.empty_like(q), torch.empty(40, Hkv, device=dev())
    qsa.paged_attn(qsa.PagedCache(k, v), batch, q, out, lse, window=W)
    K, V = (t.transpose(0, 1).reshape(Hkv, -1, D)[:, :n].double() for t in (k, v))
    rows = [0, 31, 32, 39]                                     # the items' first and last
    want, want_lse = [], []
    for r in rows:
        t = torch.arange(n, device=dev())
        z = ((K * q[r].double()[:, None]).sum(-1) * D ** -0.5).masked_fill((t > n - 40 + r) | (t <= n - 40 + r - W), float("-inf"))
        want.append((z.softmax(-1)[..., None] * V).sum(1))
        want_lse.append(torch.logsumexp(z, -1))
    out, lse, want, want_lse = out[rows], lse[rows], torch.stack(want), torch.stack(want_lse)
    # 87,000 nearly equal weights: sums within n u of |V|'s mean, here 2 (n + 40) 2^-24 0.8.
    assert (out.double() - want).abs().max() < 2 * (W + 40) * 2.0 ** -24
    assert (lse.double() - want_lse).abs().max() < (W + 40) * 2.0 ** -24 + 2e-4
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_missing_pages_are_skipped_and_reported(dtype):
    x = make_paged([200, 90], [2, 3], dtype=dtype, D=128, page=16, seed=11, poison=True)
    y = make_paged([200, 90], [2, 3], dtype=dtype, D=128, page=16, seed=11, poison=True)
    x.table[0, 3], x.table[0, 7], x.table[1, 5] = -1, 1 << 20, x.k.shape[0]
    # The reference keeps the pages and takes the tokens out of the sums: K far from every query.
    out, lse = run(x)
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "page table entries" in why
    for i, gone in ((0, {3, 7}), (1, {5})):
        K, V = y.seq_kv(i)
        r0, n, r = int(y.row_start[i]), y.lens[i], y.rows[i]
        for j in range(r):
            see = torch.tensor([t <= n - r + j and t // 16 not in gone for t in range(n)])
            for h in range(2):
                z = (y.q[r0 + j, 12 * h:12 * h + 12].double() @ K[h].nan_to_num(0.0).T) * 128 ** -0.5
                z = z.masked_fill(~see, float("-inf"))
                w = torch.softmax(z, -1)
                want = w @ V[h].nan_to_num(0.0, posinf=0.0)
                assert (out[r0 + j, 12 * h:12 * h + 12].double().cpu() - want).abs().max() < 2.0 ** -7
                assert (lse[r0 + j, 12 * h:12 * h + 12].double().cpu() - torch.logsumexp(z, -1)).abs().max() < 1e-3
    # A sequence with none of its pages sees nothing.
    x.table[0] = -1
    out, lse = run(x)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


def test_replayed_call_follows_the_lengths():
    x = make_paged([60, 500], [1, 1], dtype="bf16", D=128, page=16, seed=12)
    cache, batch, q = x.device()
    step = qsa.PagedStep(cache, batch, q, out_dtype=torch.bfloat16, window=90, n_sinks=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step.attend()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.attend()
    for lens in ([60, 500], [17, 1], [1, 321]):
        batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        step.out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        y = Paged(x.k, x.v, None, x.table, lens, [1, 1], x.row_start, x.q, 16, "head")
        assert_attended(step.out, step.lse, attend64(y, 90, 3))


def test_other_streams():
    x = make_paged([900, 400], [2, 2], dtype="bf16", D=128, page=32, seed=13)
    cache, batch, q = x.device()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    qsa.paged_attn(cache, batch, q, out, lse, stream=s)
    junk = [torch.full((1 << 20,), 3.0, device=dev()) for _ in range(4)]      # may not take the workspace over
    s.synchronize()
    assert_attended(out, lse, attend64(x))
    out.zero_()
    torch.cuda.synchronize()
    qsa.paged_attn(cache, batch, q, out, lse, stream=s.cuda_stream)
    s.synchronize()
    assert_attended(out, lse, attend64(x))
    del junk


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("D,page,order", [(128, 16, "head"), (256, 64, "token")])
def test_append_writes_the_rows_and_nothing_else(dtype, D, page, order):
    x = make_paged([5, 64, 200, 17, 40], [5, 1, 37, 0, 2], dtype=dtype, D=D, page=page, order=order, seed=20, pad_rows=3)
    cache, batch, _ = x.device()
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    fused = torch.randn(x.q.shape[0], 24 + 4, D, device=dev()).to(t)          # K and V as slices of one projection
    fused[3, 25] = 0.0                                                        # a zero row: scale 0, codes 0
    fused[6, 24:] *= 1e-6
    k_new, v_new = fused[:, 24:26], fused[:, 26:28]
    want_k, want_v = x.k.clone(), x.v.clone()
    want_s = None if x.scale is None else x.scale.clone()
    for i, (n, r) in enumerate(zip(x.lens, x.rows)):
        for j in range(r):
            p = n - r + j
            at = (int(x.table[i, p // page]), slice(None), p % page)
            row = int(x.row_start[i]) + j
            for w, (want, new) in enumerate(((want_k, k_new), (want_v, v_new))):
                if dtype == "fp8":
                    c, s = encode_fp8(new[row].float().cpu())
                    want[at], want_s[at[0], :, at[2], w] = c, s[:, 0]
                else:
                    want[at] = new[row].cpu()
    qsa.paged_append(cache, batch, k_new, v_new)
    torch.cuda.synchronize()
    assert torch.equal(cache.k.cpu(), want_k) and torch.equal(cache.v.cpu(), want_v)
    if want_s is not None:
        assert torch.equal(cache.kv_scale.cpu(), want_s)
    assert qsa.check_device_status() == (0, "")


def test_append_codes_equal_append_tokens():
    # The segment append and the paged append quantize alike.
    n, D = 9, 256
    k_new = (torch.randn(2, n, D, device=dev()) * 3).bfloat16()
    v_new = torch.randn(2, n, D, device=dev()).bfloat16()
    seg = [torch.zeros(2, 16, D, dtype=torch.uint8, device=dev()) for _ in range(2)]
    sc = torch.zeros(2, 16, 2, dtype=torch.float16, device=dev())
    idx = torch.zeros(16, 128, dtype=torch.bfloat16, device=dev())
    seq = qsa.Seq(n, n, torch.zeros(4, 128, device=dev()), [qsa.Segment(seg[0], seg[1], 0, sc)], idx_keys=idx)
    qsa.append_tokens(seq, k_new, v_new, torch.zeros(n, 128, dtype=torch.bfloat16, device=dev()))
    cache = qsa.PagedCache(*(torch.zeros(1, 2, 16, D, dtype=torch.uint8, device=dev()) for _ in range(2)),
                           torch.zeros(1, 2, 16, 2, dtype=torch.float16, device=dev()))
    one = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev())
    batch = qsa.PagedBatch(one(0)[None], one(n), one(0, n), n_rows=n)
    qsa.paged_append(cache, batch, k_new.transpose(0, 1), v_new.transpose(0, 1))
    assert torch.equal(cache.k[0], seg[0]) and torch.equal(cache.v[0], seg[1]) and torch.equal(cache.kv_scale[0], sc)


def test_append_skips_rows_without_a_page():
    x = make_paged([40], [4], dtype="bf16", D=128, page=16, seed=21)
    x.table[0, 2] = -1
    cache, batch, _ = x.device()
    new = torch.ones(4, 2, 128, dtype=torch.bfloat16, device=dev())
    before = cache.k.clone()
    qsa.paged_append(cache, batch, new, new)
    assert torch.equal(cache.k, before)
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


# ------------------------------------------------------------------ pages
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def _pool(places, each, n_pages, page, layers, dtype=torch.bfloat16, order="head", D=128, seed=0):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(layers, n_pages, 2, page, D, generator=g).to(dtype) for _ in range(2))
    put = lambda x: x.to(dev()) if order == "head" else x.to(dev()).transpose(2, 3).contiguous().transpose(2, 3)
    dk, dv = put(k), put(v)
    pool = qsa.PagePool.empty(places, each, [qsa.PagedCache(dk[i], dv[i]) for i in range(layers)])
    return pool, Pool(places, each, n_pages, page, k, v), dk, dv


def _same(pool, model, dk, dv):
    torch.cuda.synchronize()
    assert pool.lens.tolist() == model.lens
    assert pool.refs.tolist() == model.refs
    assert pool.table.tolist() == model.table
    if model.data:
        assert torch.equal(dk.cpu(), model.data[0]) and torch.equal(dv.cpu(), model.data[1])


@pytest.mark.parametrize("page,order,dtype", [(16, "head", torch.bfloat16), (64, "token", torch.float32),
                                              (32, "token", torch.bfloat16)])
@pytest.mark.parametrize("seed", range(4))
def test_random_lives_of_a_pool(page, order, dtype, seed):
    rng = random.Random(seed)
    places, each, n_pages = 9, 7, 30
    pool, model, dk, dv = _pool(places, each, n_pages, page, 3, dtype, order, seed=seed)
    qsa.check_device_status()
    for _ in range(25):
        op = rng.choice(["extend", "extend", "fork", "free", "cut", "compact"])
        n = rng.randint(1, 5)
        some = [rng.randint(-1, places) for _ in range(n)]       # out of range and repeated ones among them
        if op == "extend":
            new = [rng.choice([0, 1, rng.randint(0, 3 * page), -1]) for _ in some]
            pool.extend(_ints(some), _ints(new))
            model.extend(some, new)
        elif op == "fork":
            src = [rng.randrange(places) for _ in some]
            keep = None if rng.random() < 0.5 else [rng.randint(-1, each * page) for _ in some]
            pool.fork(_ints(src), _ints(some), None if keep is None else _ints(keep))
            model.fork(src, some, keep)
        elif op == "free":
            pool.free(_ints(some))
            model.free(some)
        elif op == "cut":
            keep = [rng.randint(-1, each * page) for _ in some]
            pool.free(_ints(some), _ints(keep))
            model.free(some, keep)
        else:
            used = _ints([-5])
            pool.compact(used)
            assert used.item() == model.compact()
        _same(pool, model, dk, dv)
    status, why = qsa.check_device_status()
    assert (status == qsa.ERR_DEVICE_CHECK and f"{model.unserved} page requests" in why) if model.unserved else status == 0


def test_pool_of_many_pages_and_requests():
    # More pages than threads, 1,024 requests, and not enough pages for the last ones.
    n_pages, places = 4000, 1100
    pool = qsa.PagePool(torch.full((places, 8), -1, dtype=torch.int32, device=dev()), _ints([0] * places),
                        _ints([0] * n_pages), page_tokens=16)
    model = Pool(places, 8, n_pages, 16)
    rng = random.Random(3)
    order = list(range(places))
    rng.shuffle(order)
    qsa.check_device_status()
    for _ in range(2):
        new = [rng.randint(0, 60) for _ in range(1024)]
        pool.extend(_ints(order[:1024]), _ints(new))
        model.extend(order[:1024], new)
        _same(pool, model, None, None)
    gone = order[100:700]
    pool.free(_ints(gone))
    model.free(gone)
    _same(pool, model, None, None)
    pool.fork(_ints(order[:100] * 5), _ints(order[100:600]))
    model.fork(order[:100] * 5, order[100:600])
    _same(pool, model, None, None)
    pool.compact()
    model.compact()
    _same(pool, model, None, None)
    assert model.unserved > 0 and qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


def test_more_caches_than_a_launch_takes():
    pool, model, dk, dv = _pool(4, 4, 12, 16, 70)
    pool.extend(_ints([2, 0]), _ints([50, 21]))
    model.extend([2, 0], [50, 21])
    pool.fork(_ints([2, 2]), _ints([1, 3]))
    model.fork([2, 2], [1, 3])
    pool.free(_ints([2]))
    model.free([2])
    pool.compact()
    model.compact()
    _same(pool, model, dk, dv)


def test_fp8_pages_move_with_their_scales():
    k = torch.randint(0, 127, (6, 2, 16, 128), dtype=torch.uint8, device=dev())
    s = torch.randn(6, 16, 2, 2, device=dev()).half().transpose(1, 2)          # scales in token order
    cache = qsa.PagedCache(k, k.flip(0).contiguous(), s)
    pool = qsa.PagePool.empty(3, 3, [cache])
    want_k, want_s = k.clone(), s.clone()
    pool.extend(_ints([0]), _ints([20]))
    pool.fork(_ints([0]), _ints([1]))                                          # page 0 shared, page 1 -> 2, 4 tokens
    want_k[2, :, :4], want_s[2, :, :4] = want_k[1, :, :4], want_s[1, :, :4]
    assert torch.equal(k, want_k) and torch.equal(s, want_s)
    pool.copy(_ints([2, 9, 4, -1]), _ints([5, 3, 4, 2]))
    want_k[5], want_s[5] = want_k[2], want_s[2]
    assert torch.equal(k, want_k) and torch.equal(s, want_s)
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK                # pages 9 and -1


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,D,window,sinks", [("bf16", 128, 0, 0), ("bf16", 256, 50, 7), ("fp8", 256, 0, 0),
                                                  ("f32", 128, 40, 2)])
def test_a_serving_run(dtype, D, window, sinks):
    """Prompt, decode, fork, decode of both, cut of a draft, free, compact, decode: every step's attention
    against 64 bits over the tokens as a plain list keeps them."""
    page, places, each, n_pages, Hkv, G = 16, 5, 12, 40, 2, 6
    g = torch.Generator().manual_seed(30)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    kind = {"bf16": torch.bfloat16, "fp8": torch.uint8, "f32": torch.float32}[dtype]
    k, v = (torch.zeros(n_pages, Hkv, page, D, dtype=kind, device=dev()) for _ in range(2))
    sc = torch.zeros(n_pages, Hkv, page, 2, dtype=torch.float16, device=dev()) if dtype == "fp8" else None
    cache = qsa.PagedCache(k, v, sc)
    pool = qsa.PagePool.empty(places, each, [cache])
    tokens = [[] for _ in range(places)]                  # (K row, V row) of each token, as stored, in 64 bits

    def stored(x):
        if dtype != "fp8":
            return x.double()
        c, s = encode_fp8(x.float())
        return c.view(torch.float8_e4m3fn).double() * s.double()

    def step(who, counts):
        n = sum(counts)
        k_new, v_new = (torch.randn(n, Hkv, D, generator=g).to(act) for _ in range(2))
        q = (torch.randn(n, Hkv * G, D, generator=g) * 2).to(act)
        pool.extend(_ints(who), _ints(counts))
        rows = [counts[who.index(s)] if s in who else 0 for s in range(places)]
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        by_place = [who.index(s) for s in range(places) if s in who]
        at = [0]
        for c in counts:
            at.append(at[-1] + c)
        perm = [j for w in by_place for j in range(at[w], at[w + 1])]
        k_new, v_new, q = k_new[perm], v_new[perm], q[perm]
        for s in range(places):
            for j in range(starts[s], starts[s + 1]):
                tokens[s].append((stored(k_new[j]), stored(v_new[j])))
        batch = qsa.PagedBatch(pool.table, pool.lens, _ints(starts), n_rows=n, max_rows=max(rows))
        st = qsa.PagedStep(cache, batch, q.to(dev()), window=window, n_sinks=sinks)
        out, lse = st.run(k_new.to(dev()), v_new.to(dev()))
        torch.cuda.synchronize()
        assert pool.lens.tolist() == [len(t) for t in tokens]
        L = max(len(t) for t in tokens)
        plain = Paged(torch.zeros(places, Hkv, L, D, dtype=torch.float64), torch.zeros(places, Hkv, L, D, dtype=torch.float64),
                      None, torch.arange(places, dtype=torch.int32)[:, None], [len(t) for t in tokens], rows,
                      torch.tensor(starts), q, L, "head")
        for s in range(places):
            for t, (a, b) in enumerate(tokens[s]):
                plain.k[s, :, t], plain.v[s, :, t] = a, b
        assert_attended(out, lse, attend64(plain, window, sinks))

    step([3, 0], [70, 33])                                # prompts
    step([0, 3], [1, 1])
    pool.fork(_ints([3, 0]), _ints([1, 4]))
    tokens[1], tokens[4] = list(tokens[3]), list(tokens[0])
    step([0, 1, 3, 4], [1, 4, 2, 1])                      # four rows of a draft for sequence 1 ...
    pool.free(_ints([1]), _ints([len(tokens[1]) - 3]))    # ... of which one is kept
    tokens[1] = tokens[1][:-3]
    pool.free(_ints([3]))
    tokens[3] = []
    step([1, 4], [1, 1])
    used = _ints([0])
    pool.compact(used)
    assert used.item() == len({int(p) for s in range(places) for p in pool.table[s, :-(-len(tokens[s]) // page)].tolist()})
    step([0, 1, 3, 4], [1, 1, 20, 2])
    assert qsa.check_device_status() == (0, "")


def test_runs_of_many_windowed_items():
    # Runs that hold several items of several tiles each, with and without first tokens apart from the window.
    x = make_paged([900 + 37 * i for i in range(40)], [1] * 40, dtype="bf16", Hkv=2, G=2, page=32, seed=40)
    for n in (3, 0):
        check(x, window=600, sinks=4, n_splits=n)
        check(x, window=300, n_splits=n)
