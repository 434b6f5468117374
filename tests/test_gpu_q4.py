"""Attention over 4-bit paged caches against 64 bits, their pages, and runs of
rotation, append and attention together.  Tolerances are derived in q4_cases."""
import math
import random

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import assert_attended, dev
from q4_cases import Paged4, attend4, encode4, make_paged4, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    qsa.check_device_status()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def run(x, *, out_dtype=torch.float32, window=0, sinks=0, n_splits=0, scale=0.0):
    cache, batch, q = x.device()
    out = torch.full(q.shape, 7.0, dtype=out_dtype, device=dev())
    lse = torch.full(q.shape[:2], 7.0, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse, window=window, n_sinks=sinks, n_splits=n_splits, scale=scale)
    torch.cuda.synchronize()
    return out, lse


def check(x, **kw):
    ref = attend4(x, kw.get("window", 0), kw.get("sinks", 0), kw.get("scale") or None)
    out, lse = run(x, **kw)
    assert_attended(out, lse, ref, sum(x.rows))
    assert qsa.check_device_status() == (0, "")
    return out, lse


@pytest.mark.parametrize("D", [128, 256])
def test_one_key(D):
    # One token: the output is its V, whatever the logit.
    x = make_paged4([1], [1], D=D, page=16, seed=1, Hkv=1, G=1)
    check(x)


@pytest.mark.parametrize("D,page,order", [(128, 16, "head"), (256, 32, "token"), (256, 64, "head"), (128, 256, "token")])
@pytest.mark.parametrize("rows", [[1] * 13, [1, 2, 1, 4, 3, 1, 1, 2, 1, 8, 5, 1, 2]])
def test_decode_and_verify_ragged(D, page, order, rows):
    # Lengths of one, around page and tile ends, and long enough to be split.
    x = make_paged4([1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700, 2049], rows, D=D, page=page, order=order, seed=1, poison=True)
    check(x)


@pytest.mark.parametrize("D,rows", [(128, [1, 1, 1, 1, 1]), (128, [1, 2, 9, 1, 30]), (256, [1, 1, 1, 1, 1]), (256, [1, 2, 9, 1, 30])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 0), (100, 5), (128, 64), (129, 128), (500, 130),
                                          (1 << 30, 9), (200, 1 << 30)])
def test_windows_and_sinks(D, rows, window, sinks):
    x = make_paged4([1, 40, 300, 777, 1025], rows, D=D, page=32, seed=2, poison=True)
    check(x, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 10)])
def test_chunks_of_rows(D, window, sinks):
    x = make_paged4([400, 333, 90], [300, 65, 90], D=D, page=64, seed=3, poison=True)
    check(x, window=window, sinks=sinks, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (8, 1), (3, 5), (1, 16), (4, 8), (2, 7)])
@pytest.mark.parametrize("rows", [[2, 17, 1], [1, 1, 1]])
def test_head_layouts(Hkv, G, rows):
    x = make_paged4([130, 40, 300], rows, D=128, Hkv=Hkv, G=G, page=32, seed=4, poison=True)
    check(x)
    check(x, window=33, sinks=2, scale=0.3)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 512, 1024])
def test_page_sizes(page):
    check(make_paged4([1500, 3, 129], [1, 1, 1], D=256, page=page, seed=page, poison=True))
    check(make_paged4([1500, 3, 129], [4, 2, 3], D=128, page=page, order="token", seed=page, poison=True), window=300, sinks=20)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("rows", [[2], [1]])
def test_tokens_outside_the_window_may_hold_anything(D, rows):
    # Everything before the window and behind the sinks: records of NaN and infinities.
    W, S, n, r = 100, 20, 600, rows[0]
    x = make_paged4([n], [r], D=D, page=16, seed=5, poison=True)
    for t in range(S, n - r - W + 1):
        p, s = int(x.table[0, t // 16]), t % 16
        x.k[p, :, s], x.v[p, :, s] = 0xFF, 0x80
        x.scale[p, :, s] = torch.tensor([math.nan, -math.inf, math.inf, math.nan] * (D // 32), dtype=torch.float16)
    check(x, window=W, sinks=S)


def test_rows_that_see_nothing_and_rows_of_nobody():
    x = make_paged4([50, 0, 30, 3], [2, 0, 0, 3], D=128, page=16, seed=6, pad_rows=5)
    cache, batch, q = x.device()
    start = _ints([1, 3, 4, 4, 9])                         # 1: no tokens but a row; 3: 3 tokens and 5 rows
    batch = qsa.PagedBatch(batch.table, batch.lens, start, n_rows=q.shape[0], max_rows=5)
    out, lse = torch.full(q.shape, 7.0, device=dev()), torch.full(q.shape[:2], 7.0, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse)
    y = Paged4(x.k, x.v, x.scale, x.table, [50, 0, 30, 3], [2, 0, 0, 3], torch.tensor([1, 3, 3, 3, 6]), None, 16, "head")
    y.q = torch.cat((x.q[:3], x.q[6:9]))
    keep = [1, 2, 6, 7, 8]
    assert_attended(out[keep], lse[keep], tuple(t[[1, 2, 3, 4, 5]] for t in attend4(y, most=5)))
    for r in (3, 4, 5):
        assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    for r in (0, 9):
        assert (out[r] == 7).all() and (lse[r] == 7).all()
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("most", [1, 2])
def test_more_rows_than_promised(D, most):
    # Items then end inside a row's heads (16 entries of 12 heads), or there are several of whole rows.
    x = make_paged4([400, 90, 33], [5, 1, 33], D=D, Hkv=2, G=12, page=32, seed=25)
    cache, batch, q = x.device()
    batch = qsa.PagedBatch(batch.table, batch.lens, batch.row_start, n_rows=q.shape[0], max_rows=most)
    for window, sinks in ((0, 0), (20, 3)):
        out, lse = torch.empty(q.shape, device=dev()), torch.empty(q.shape[:2], device=dev())
        qsa.paged_attn(cache, batch, q, out, lse, window=window, n_sinks=sinks)
        assert_attended(out, lse, attend4(x, window, sinks, most=most))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("rows", [[1, 1, 1], [4, 1, 2]])
def test_divisions_agree_and_repeat(D, rows):
    x = make_paged4([3000, 70, 900], rows, D=D, page=64, seed=7)
    ref = attend4(x)
    for n in (1, 2, 3, 7, 50, 0):
        out, lse = run(x, n_splits=n)
        assert_attended(out, lse, ref)
        for _ in range(5):
            again, lse2 = run(x, n_splits=n)
            assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("most", [1, 3])
def test_one_run_of_short_items(D, most):
    lens = [1 + (37 * i) % 390 for i in range(40)]
    x = make_paged4(lens, [1 + i % most if n > 3 else 1 for i, n in enumerate(lens)], D=D, page=32, seed=33)
    for n in (1, 2, 5):
        first = check(x, n_splits=n)
        for _ in range(5):
            again = run(x, n_splits=n)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_outputs_and_workspaces_on_16_bytes(out_dtype):
    x = make_paged4([700, 9, 40], [4, 1, 40], D=128, page=64, seed=14)
    cache, batch, q = x.device()
    cfg = cache.config(24, out_dtype)
    ws = torch.empty(qsa.paged_attn_workspace_size(batch, cfg) + 16, dtype=torch.uint8, device=dev())[16:]
    es = torch.empty(0, dtype=out_dtype).element_size()
    out = torch.empty(q.numel() + 16 // es, dtype=out_dtype, device=dev())[16 // es:].view(q.shape)
    q2 = torch.empty(q.numel() + 8, dtype=q.dtype, device=dev())[8:].view(q.shape)
    q2.copy_(q)
    lse = torch.empty(q.numel() // 128 + 1, device=dev())[1:].view(q.shape[:2])
    assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    qsa.paged_attn(cache, batch, q2, out, lse, workspace=ws, cfg=cfg)
    assert_attended(out, lse, attend4(x))


@pytest.mark.parametrize("n,chunks", [(700, {}), (130, {129: 290, 70: 9}), (420, {3: 280, 200: 37, 401: 300, 419: 5})])
def test_many_sequences(n, chunks):
    rng = random.Random(n)
    lens = [rng.randint(1, 90) for _ in range(n)]
    rows = [rng.choice([0, 1, 1, 2]) if m > 1 else 1 for m in lens]
    for i, r in chunks.items():
        lens[i], rows[i] = r + rng.randint(0, 200), r
    x = make_paged4(lens, rows, D=128, Hkv=1, G=4, page=16, seed=n, poison=True)
    check(x)
    check(x, window=20, sinks=2)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("rows", [[1, 1], [3, 12]])
def test_queries_of_any_size(D, rows):
    # Rows of queries from 1e-30 to 1e30 beside each other, and channels far apart in one row.
    x = make_paged4([300, 90], rows, D=D, Hkv=1, G=4, page=16, seed=15)
    q = x.q.float()
    flat = q.view(-1, D)
    flat[0] *= 1e-30
    flat[1] = 0.0
    flat[2, 5] *= 1000.0
    flat[3] *= torch.logspace(-12, 0, D)
    x.q = q.bfloat16()
    check(x)
    x.q = x.q * 1e30
    check(x, scale=D ** -0.5 * 1e-30)


def test_queries_that_are_no_numbers_stay_in_their_rows():
    for rows in ([1, 1], [9, 1]):
        x = make_paged4([200, 60], rows, D=128, Hkv=1, G=4, page=16, seed=16)
        clean, _ = run(x)
        x.q[0, 1, 7], x.q[-1, 3, 0] = float("nan"), float("inf")
        out, lse = run(x)
        bad = torch.zeros(out.shape[:2], dtype=torch.bool)
        bad[0, 1] = bad[-1, 3] = True
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("rows", [[2, 1, 1], [1, 1, 1], [20, 6, 6]])
def test_scales_of_any_size(D, rows):
    # V of very different sizes by token and block, scales that are negative, zero, subnormal and the largest.
    x = make_paged4([500, 40, 300], rows, D=D, page=32, seed=17)
    G = D // 32
    rec = x.scale.view(*x.scale.shape[:3], 2, G, 2).float()
    g = torch.Generator().manual_seed(17)
    rec[..., 1, :, 0] *= 10.0 ** (torch.rand(rec.shape[:3] + (G,), generator=g) * 8 - 6)
    rec[..., 1, 0, 0] *= -1.0
    rec[..., 1, 1, 0] = 0.0
    rec[..., 0, 1, 0] *= -0.5
    rec[..., 0, 2, 0] = 2.0 ** -24
    rec[..., 1, 3, :] *= 1e-4
    rec[..., 1, :, :].clamp_(-2000.0, 2000.0)              # (values have to lie within f16's range)
    for t, s in ((7, 4000.0), (123, 3000.0), (400, -4000.0)):
        rec[x.table[0, t // 32], 0, t % 32, 1, 2, 0] = s
    x.scale = rec.half().view(x.scale.shape)
    check(x)


def test_logits_that_climb():
    # Every tile's logits are above the last one's: the maximum moves all the time, and once by a lot.
    for rows, D in (([1], 256), ([5], 128), ([9], 128), ([8], 256)):
        x = make_paged4([1500], rows, D=D, Hkv=1, G=3, page=64, seed=18, lean=0.0)
        x.q[:] = 0.0
        x.q[..., 0] = torch.linspace(1.0, 3.0, 3)[None].bfloat16()
        rec = x.scale.view(*x.scale.shape[:3], 2, D // 32, 2)
        for t in range(1500):
            rec[x.table[0, t // 64], 0, t % 64, 0, 0] = torch.tensor([0.01, t * 0.4 + (300.0 if t > 900 else 0.0)], dtype=torch.float16)
        check(x)
        check(x, window=700, sinks=30)


def test_pages_past_32_bits():
    # Byte offsets above 2^32: page 60,000 of 64 tokens x 2 heads x 768 bytes.
    page, n_pages = 64, 60_002
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 14 GB")
    x = make_paged4([100], [2], D=256, page=page, seed=10)
    k, v = (torch.empty(n_pages, 2, page, 768, dtype=torch.uint8, device=dev())[..., :128] for _ in range(2))
    sc = torch.empty(n_pages, 2, page, 32, dtype=torch.float16, device=dev())
    at = [60_001, 59_999]
    for j, p in enumerate(at):
        k[p], v[p], sc[p] = (y[x.table[0, j]].to(dev()) for y in (x.k, x.v, x.scale))
    batch = qsa.PagedBatch(_ints([at]), _ints([100]), _ints([0, 2]), n_rows=2)
    cache, q = qsa.PagedCache(k, v, sc, kv_dtype=qsa.Q4), x.q.to(dev())
    out, lse = torch.empty(2, 24, 256, device=dev()), torch.empty(2, 24, device=dev())
    qsa.paged_attn(cache, batch, q, out, lse)
    assert_attended(out, lse, attend4(x))
    new = torch.randn(2, 2, 256, device=dev()).bfloat16()
    qsa.paged_append(cache, batch, new, new)
    back = [torch.empty(2, 2, 256, device=dev()) for _ in range(2)]
    qsa.paged_read(cache, batch, *back)
    assert torch.equal(k[59_999, :, 34:36].cpu(), encode4(new.cpu().float())[0].transpose(0, 1))
    assert (back[0] - new.float()).abs().max() < 0.5 and torch.equal(back[0], back[1])
    pool = qsa.PagePool(batch.table, batch.lens, torch.zeros(n_pages, dtype=torch.int32, device=dev()), [cache])
    pool.copy(_ints([60_001]), _ints([59_000]))
    assert torch.equal(k[59_000], k[60_001]) and torch.equal(sc[59_000], sc[60_001])


def test_lengths_at_the_ends_of_32_bits():
    x = make_paged4([40, 40], [3, 2], D=128, seed=41)
    cache, batch, q = x.device()
    out, lse = torch.full(q.shape, 7.0, device=dev()), torch.full(q.shape[:2], 7.0, device=dev())
    batch.lens[0] = 2 ** 31 - 1
    qsa.paged_attn(cache, batch, q, out, lse, window=64, n_sinks=40)
    torch.cuda.synchronize()
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK
    K, V = x.seq_kv(0)
    z = torch.einsum("rhgd,htd->rhgt", x.q[:3].double().view(3, -1, 12, 128), K) * 128 ** -0.5
    want = torch.einsum("rhgt,htd->rhgd", z.softmax(-1), V).reshape(3, -1, 128)
    assert (out[:3].double().cpu() - want).abs().max() < 2.0 ** -9 * 2 * V.abs().max()   # three roundings of weights to f16
    batch.lens[0] = 1                                      # rows at positions -2, -1 and 0
    for window in (0, 2 ** 31 - 1, 2 ** 31 - 2 ** 26):
        qsa.paged_attn(cache, batch, q, out, lse, window=window)
        torch.cuda.synchronize()
        assert (out[:2] == 0).all() and torch.isinf(lse[:2]).all() and torch.isfinite(lse[2:5]).all()
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("D,rows", [(128, [2, 3]), (256, [1, 1])])
def test_missing_pages_are_skipped_and_reported(D, rows):
    x = make_paged4([200, 90], rows, D=D, page=16, seed=11, poison=True)
    full = x.table.clone()
    x.table[0, 3], x.table[0, 7], x.table[1, 5] = -1, 1 << 20, x.k.shape[0]
    out, lse = run(x)
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "page table entries" in why
    x.table = full
    for i, gone in ((0, {3, 7}), (1, {5})):
        K, V = x.seq_kv(i)
        r0, n, r = int(x.row_start[i]), x.lens[i], x.rows[i]
        for j in range(r):
            see = torch.tensor([t <= n - r + j and t // 16 not in gone for t in range(n)])
            for h in range(2):
                z = (x.q[r0 + j, 12 * h:12 * h + 12].double() @ K[h].T) * D ** -0.5
                z = z.masked_fill(~see, float("-inf"))
                assert (out[r0 + j, 12 * h:12 * h + 12].double().cpu() - torch.softmax(z, -1) @ V[h]).abs().max() < 2.0 ** -7
                assert (lse[r0 + j, 12 * h:12 * h + 12].double().cpu() - torch.logsumexp(z, -1)).abs().max() < 1e-3
    x.table = full.clone()
    x.table[0] = -1
    out, lse = run(x)
    r = x.rows[0]
    assert (out[:r] == 0).all() and torch.isneginf(lse[:r]).all()
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


@pytest.mark.parametrize("rows", [[1, 1], [2, 17]])
def test_replayed_call_follows_the_lengths(rows):
    x = make_paged4([60, 500], rows, D=128, page=16, seed=12)
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
    for lens in ([60, 500], [17, 17], [2, 321]):
        batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        step.out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        y = Paged4(x.k, x.v, x.scale, x.table, lens, rows, x.row_start, x.q, 16, "head")
        assert_attended(step.out, step.lse, attend4(y, 90, 3))


def test_steps_at_once_on_two_streams():
    # Two steps over one cache, each with a workspace of its own, many times at once.
    x = make_paged4([3000, 700], [1, 3], D=256, page=32, seed=13)
    cache, batch, q = x.device()
    steps = [qsa.PagedStep(cache, batch, q, window=w, n_sinks=5) for w in (0, 300)]
    refs = [attend4(x, w, 5) for w in (0, 300)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, s in zip(steps, streams):
            st.attend(s)
    torch.cuda.synchronize()
    for st, ref in zip(steps, refs):
        assert_attended(st.out, st.lse, ref)


# ------------------------------------------------------------------ pages
def test_pages_move_with_their_records():
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randint(0, 256, (6, 2, 16, 64), dtype=torch.uint8, device=dev(), generator=g)
    s = torch.randn(6, 16, 2, 16, device=dev(), generator=g).half().transpose(1, 2)   # records in token order
    cache = qsa.PagedCache(k, k.flip(0).contiguous(), s, kv_dtype=qsa.Q4)
    pool = qsa.PagePool.empty(3, 3, [cache])
    want_k, want_v, want_s = k.clone(), cache.v.clone(), s.clone()
    pool.extend(_ints([0]), _ints([20]))
    pool.fork(_ints([0]), _ints([1]))                      # page 0 shared, page 1 -> 2, 4 tokens
    for y in (want_k, want_v, want_s):
        y[2, :, :4] = y[1, :, :4]
    assert torch.equal(k, want_k) and torch.equal(cache.v, want_v) and torch.equal(s, want_s)
    pool.copy(_ints([2, 9, 4, -1]), _ints([5, 3, 4, 2]))
    for y in (want_k, want_v, want_s):
        y[5] = y[2]
    assert torch.equal(k, want_k) and torch.equal(cache.v, want_v) and torch.equal(s, want_s)
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK     # pages 9 and -1


@pytest.mark.parametrize("D,order", [(128, "head"), (256, "token")])
def test_compact_moves_records(D, order):
    cache = qsa.PagedCache.zeros(12, 2, 16, D, qsa.Q4)
    for t in (cache.k, cache.v):
        t.copy_(torch.arange(12, device=dev(), dtype=torch.uint8)[:, None, None, None].expand_as(t))
    cache.kv_scale.copy_(torch.arange(12, device=dev()).half()[:, None, None, None].expand_as(cache.kv_scale))
    pool = qsa.PagePool.empty(3, 4, [cache])
    pool.extend(_ints([0, 1, 2]), _ints([50, 40, 60]))
    pool.free(_ints([0]))
    was = pool.table.clone()
    used = _ints([0])
    pool.compact(used)
    assert used.item() == 7
    for s, n in ((1, 3), (2, 4)):
        for j in range(n):
            new, old = int(pool.table[s, j]), int(was[s, j])
            assert new < 7 and (cache.k[new] == old).all() and (cache.v[new] == old).all() and (cache.kv_scale[new] == old).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,window,sinks,rot,pairs", [(128, 0, 0, 128, False), (256, 50, 7, 64, True)])
def test_a_serving_run_with_rotation(D, window, sinks, rot, pairs):
    """Prompt, decode, fork, decode of both, free, compact, decode, with rotated rows in 4 bits: every step's attention
    against 64 bits over the tokens as a plain list keeps them, and the rows read back."""
    page, places, each, n_pages, Hkv, G = 16, 5, 12, 40, 2, 6
    g = torch.Generator().manual_seed(30)
    cache = qsa.PagedCache.zeros(n_pages, Hkv, page, D, qsa.Q4)
    pool = qsa.PagePool.empty(places, each, [cache])
    rope = qsa.Rope(rot, base=1e5, pairs=pairs, scaling=qsa.RopeScaling("linear", 2.0))
    tokens = [[] for _ in range(places)]                   # (K codes, K pairs, V codes, V pairs) of each token

    def step(counts):
        n = sum(counts)
        fused = torch.randn(n, Hkv * (G + 2), D, generator=g).bfloat16()
        q, k_new, v_new = fused[:, :Hkv * G] * 2, fused[:, Hkv * G:Hkv * (G + 1)], fused[:, Hkv * (G + 1):]
        who = [s for s in range(places) if counts[s]]
        pool.extend(_ints(who), _ints([counts[s] for s in who]))
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + c)
        pos = [len(tokens[s]) + j for s in range(places) for j in range(counts[s])]
        # The rotated rows as the rotation by itself leaves them (tested against 64 bits elsewhere).
        k_rot, q_rot = (qsa.rotate(rope, _ints(pos), y.to(dev()).contiguous()).cpu() for y in (k_new, q))
        assert (k_rot.double() - turned(k_new, pos, rot, pairs, rope.frequencies)).abs().max() < 2.0 ** -8 * 6
        for s in range(places):
            for j in range(starts[s], starts[s + 1]):
                tokens[s].append((*encode4(k_rot[j].float()), *encode4(v_new[j].float())))
        batch = qsa.PagedBatch(pool.table, pool.step_lens, _ints(starts), n_rows=n, max_rows=max(counts))
        st = qsa.PagedStep(cache, batch, q.to(dev()), window=window, n_sinks=sinks, rope=rope)
        out, lse = st.run(k_new.to(dev()), v_new.to(dev()))
        torch.cuda.synchronize()
        assert pool.lens.tolist() == [len(t) for t in tokens] and torch.equal(st.q_rotated.cpu(), q_rot)
        L = max(len(t) for t in tokens)
        z8 = torch.zeros(places, Hkv, L, D // 2, dtype=torch.uint8)
        plain = Paged4(z8, z8.clone(), torch.zeros(places, Hkv, L, D // 8, dtype=torch.float16),
                       torch.arange(places, dtype=torch.int32)[:, None], [len(t) for t in tokens], list(counts),
                       torch.tensor(starts), q_rot, L, "head")
        for s in range(places):
            for t, (kc, kp, vc, vp) in enumerate(tokens[s]):
                plain.k[s, :, t], plain.v[s, :, t] = kc, vc
                plain.scale[s, :, t] = torch.cat((kp.flatten(-2), vp.flatten(-2)), -1)
        assert_attended(out, lse, attend4(plain, window, sinks))
        back = [torch.empty(n, Hkv, D, device=dev()) for _ in range(2)]
        qsa.paged_read(cache, batch, *back)
        want = [torch.cat([plain.seq_kv(s)[w][:, -c:].transpose(0, 1) for s, c in enumerate(counts) if c]) for w in range(2)]
        for a, b in zip(back, want):
            assert (a.double().cpu() - b).abs().max() <= 2.0 ** -23 * b.abs().max()

    step([33, 0, 0, 70, 0])                                # prompts
    step([1, 0, 0, 1, 0])
    pool.fork(_ints([3, 0]), _ints([1, 4]))
    tokens[1], tokens[4] = list(tokens[3]), list(tokens[0])
    step([1, 4, 0, 2, 1])                                  # four rows of a draft for sequence 1 ...
    pool.free(_ints([1]), _ints([len(tokens[1]) - 3]))     # ... of which one is kept
    tokens[1] = tokens[1][:-3]
    pool.free(_ints([3]))
    tokens[3] = []
    step([0, 1, 0, 0, 1])
    pool.compact()
    step([1, 1, 0, 20, 2])
    assert qsa.check_device_status() == (0, "")


def test_a_step_with_a_rope_takes_new_rows():
    x = make_paged4([40], [1], D=128, page=16, seed=26)
    cache, batch, q = x.device()
    st = qsa.PagedStep(cache, batch, q, rope=qsa.Rope(64))
    with pytest.raises(ValueError, match="new rows"):
        st.run()
    rows = torch.zeros(1, cache.n_kv_heads, 128, dtype=torch.bfloat16, device=dev())
    out, lse = st.run(rows, rows)
    again, lse2 = (t.clone() for t in (out, lse))
    assert torch.equal(st.attend()[0], again) and torch.equal(lse, lse2)
