"""Rotations on the GPU, by themselves and on the way into a paged cache, and rows
read back out of their pages.  Tolerances are derived in q4_cases."""
import math

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import dev, encode_fp8, make_paged
from q4_cases import assert_turned, encode4, make_paged4, split4, turned

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


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rows,heads,D,rot", [(1, 1, 16, 16), (7, 24, 128, 128), (33, 3, 256, 64), (5, 24, 256, 256),
                                              (3, 2, 1024, 256), (130, 1, 48, 32), (2, 40, 128, 112)])
def test_rotation(dtype, pairs, rows, heads, D, rot):
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, heads, D, generator=g) * 3).to(dtype)
    pos = torch.randint(0, 300_000, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 0
    for scaling in (None, qsa.RopeScaling("linear", 7.5), qsa.RopeScaling("parts", 32.0, original_tokens=8192)):
        r = qsa.Rope(rot, base=1e6, pairs=pairs, scaling=scaling)
        xd = x.to(dev())
        out = torch.full_like(xd, 5.0)
        assert qsa.rotate(r, pos.to(dev()), xd, out) is out
        assert_turned(out, x, pos, rot, pairs, r.frequencies, r.magnitude)
        assert torch.equal(out[..., rot:].cpu(), x[..., rot:]) and torch.equal(xd.cpu(), x)
        assert qsa.rotate(r, pos.to(dev()), xd) is xd and torch.equal(xd, out)      # in place: the same bits


@pytest.mark.parametrize("pairs", [False, True])
def test_far_and_negative_positions(pairs):
    # The angle of a position is reduced exactly: far ones keep their precision, negative ones turn back.
    D = 128
    x = torch.randn(6, 2, D)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 1, 1 << 30, 12_345_678], dtype=torch.int32)
    w = [2 * math.pi * k / 64 for k in range(D // 2)]     # whole turns every 64 positions
    r = qsa.Rope(D, frequencies=w, pairs=pairs)
    got = qsa.rotate(r, pos.to(dev()), x.to(dev()), torch.empty(6, 2, D, device=dev()))
    assert_turned(got, x, pos.long() % 64, D, pairs, w, farthest=2.0 ** 31)
    # (-2^31 has no opposite: its row is left out.)
    back = qsa.rotate(r, (-pos).to(dev()), got.clone())
    keep = [0, 2, 3, 4, 5]
    assert (back.cpu() - x)[keep].abs().max() < 40 * 2.0 ** -24 * x.abs().max()


def test_rotation_of_strided_rows_and_heads():
    # Slices of one projection into token-major and head-major outputs, odd addresses of 16 bytes.
    fused = torch.randn(9, 30, 128, device=dev()).bfloat16()
    pos = torch.arange(100, 109, dtype=torch.int32, device=dev())
    r = qsa.Rope(64, pairs=True)
    want = qsa.rotate(r, pos, fused[:, 3:8].contiguous())
    for out in (torch.zeros(9, 12, 128, device=dev()).bfloat16()[:, 5:10],
                torch.zeros(5, 9, 128, device=dev()).bfloat16().transpose(0, 1),
                torch.zeros(9, 5, 160, device=dev()).bfloat16()[..., 8:136]):
        qsa.rotate(r, pos, fused[:, 3:8], out)
        assert torch.equal(out, want)
    rest = fused[:, [0, 1, 2, 8, 9]].clone()
    qsa.rotate(r, pos, fused[:, 3:8])                      # in place inside the projection
    assert torch.equal(fused[:, 3:8], want) and torch.equal(fused[:, [0, 1, 2, 8, 9]], rest)
    one = torch.randn(1, 1, 128, device=dev())
    assert torch.equal(qsa.rotate(r, pos[:1], one[:, :, :].clone()), qsa.rotate(r, pos[:1], one.expand(1, 1, 128).clone()))
    empty = torch.empty(0, 5, 128, device=dev())
    qsa.rotate(r, pos[:0], empty)


def test_rotation_keeps_what_is_no_number_in_its_pair():
    x = torch.randn(2, 1, 64, device=dev())
    x[0, 0, 3], x[1, 0, 40] = float("nan"), float("inf")
    got = qsa.rotate(qsa.Rope(64), _ints([5, 6]), x, torch.empty_like(x))
    bad = ~torch.isfinite(got)
    assert bad[0, 0].nonzero().flatten().tolist() == [3, 35] and set(bad[1, 0].nonzero().flatten().tolist()) <= {8, 40}


def test_rotation_on_other_streams_and_replayed():
    x = torch.randn(50, 4, 128, device=dev()).bfloat16()
    pos, r = torch.arange(50, dtype=torch.int32, device=dev()), qsa.Rope(128)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qsa.rotate(r, pos, x, out, stream=s)
    s.synchronize()
    assert_turned(out, x.cpu(), pos.cpu(), 128, False, r.frequencies)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qsa.rotate(r, pos, x, out)
    for shift in (7, 100_000):
        pos += shift
        graph.replay()
        torch.cuda.synchronize()
        assert_turned(out, x.cpu(), pos.cpu(), 128, False, r.frequencies)


# ------------------------------------------------------------------ append
def _state(dtype, lens, rows, **kw):
    x = make_paged4(lens, rows, **kw) if dtype == "q4" else make_paged(lens, rows, dtype=dtype, **kw)
    return x, *x.device()


def _encoded(dtype, row):
    """What a cache holds of [heads, D] rows: codes or values, and records."""
    if dtype == "q4":
        c, p = encode4(row.float())
        return c, p.flatten(-2)
    return encode_fp8(row.float()) if dtype == "fp8" else (row, None)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32", "q4"])
@pytest.mark.parametrize("D,page,order,rot,pairs", [(128, 16, "head", 128, False), (256, 64, "token", 256, False),
                                                    (256, 16, "head", 64, True), (128, 32, "token", 48, False),
                                                    (128, 16, "head", 0, False)])
def test_append_with_rotation(dtype, D, page, order, rot, pairs):
    """The same bits as the rotation by itself and an append; rows, pages and queries of nobody as they were."""
    if rot == 0 and dtype != "q4":
        pytest.skip("the plain append, tested with the other caches")
    lens, rows = [5, 64, 200, 17, 40], [5, 1, 37, 0, 2]
    x, cache, batch, _ = _state(dtype, lens, rows, D=D, page=page, order=order, seed=20, pad_rows=3)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    n = x.q.shape[0]
    fused = torch.randn(n, 24 + 4, D, device=dev()).to(t)
    fused[3, 25] = 0.0                                     # a row of zeros, a constant one, a tiny one
    fused[4, 26] = 1.5
    fused[6, 24:] *= 1e-6
    q, k_new, v_new = fused[:, :24], fused[:, 24:26], fused[:, 26:28]
    before = fused.clone()
    pos = torch.zeros(n, dtype=torch.int32)
    for i, (m, r) in enumerate(zip(lens, rows)):
        for j in range(r):
            pos[int(x.row_start[i]) + j] = m - r + j
    q_out = torch.full((n, 24, D), 9.0, dtype=t, device=dev())
    if rot:
        rope = qsa.Rope(rot, base=1e5, pairs=pairs, scaling=qsa.RopeScaling("parts", 4.0, original_tokens=64))
        turned_k = qsa.rotate(rope, pos.to(dev()), k_new, torch.empty(n, 2, D, dtype=t, device=dev()))
        turned_q = qsa.rotate(rope, pos.to(dev()), q, torch.empty(n, 24, D, dtype=t, device=dev()))
        assert_turned(turned_k, k_new.cpu(), pos, rot, pairs, rope.frequencies, rope.magnitude)
        qsa.paged_append(cache, batch, k_new, v_new, rope=rope, q=q, q_out=q_out)
    else:
        turned_k = k_new
        qsa.paged_append(cache, batch, k_new, v_new)
    torch.cuda.synchronize()
    want_k, want_v = x.k.clone(), x.v.clone()
    want_s = None if x.scale is None else x.scale.clone()
    used = sum(rows)
    for i, (m, r) in enumerate(zip(lens, rows)):
        for j in range(r):
            row, p = int(x.row_start[i]) + j, m - r + j
            at = (int(x.table[i, p // page]), slice(None), p % page)
            for w, (want, new) in enumerate(((want_k, turned_k), (want_v, v_new))):
                c, s = _encoded(dtype, new[row].cpu())
                want[at] = c
                if s is not None:
                    half = s.shape[-1]
                    want_s[at[0], :, at[2], w * half:(w + 1) * half] = s
    assert torch.equal(cache.k.cpu(), want_k) and torch.equal(cache.v.cpu(), want_v)
    if want_s is not None:
        assert torch.equal(cache.kv_scale.cpu(), want_s)
    assert torch.equal(fused, before)
    if rot:
        assert torch.equal(q_out[:used], turned_q[:used]) and (q_out[used:] == 9).all()
        again = q.contiguous()                             # queries in place, and none at all
        qsa.paged_append(cache, batch, k_new, v_new, rope=rope, q=again, q_out=again)
        assert torch.equal(again[:used], turned_q[:used]) and torch.equal(again[used:], q[used:])
        cache.k.zero_()
        qsa.paged_append(cache, batch, k_new, v_new, rope=rope)
        at = (int(x.table[0, 0]), slice(None), 0)
        assert torch.equal(cache.k[at].cpu(), want_k[at])
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "q4"])
def test_append_of_many_heads_and_few(dtype):
    # More K and V rows than a CTA has warps; one head of each; no queries.
    for Hkv, G in ((17, 1), (1, 16), (5, 3)):
        x, cache, batch, _ = _state(dtype, [30, 9], [3, 9], D=128, Hkv=Hkv, G=G, page=16, seed=Hkv)
        k_new, v_new = (torch.randn(12, Hkv, 128, device=dev()).bfloat16() for _ in range(2))
        q = torch.randn(12, Hkv * G, 128, device=dev()).bfloat16()
        rope, pos = qsa.Rope(128), _ints([27, 28, 29, *range(9)])
        q_out = torch.empty_like(q)
        qsa.paged_append(cache, batch, k_new, v_new, rope=rope, q=q, q_out=q_out)
        assert torch.equal(q_out, qsa.rotate(rope, pos, q.clone()))
        k = qsa.rotate(rope, pos, k_new.clone()).cpu()
        for row, (i, p) in enumerate([(0, 27), (0, 28), (0, 29), *((1, p) for p in range(9))]):
            at = (int(x.table[i, p // 16]), slice(None), p % 16)
            assert torch.equal(cache.k[at].cpu(), _encoded(dtype, k[row])[0])
            assert torch.equal(cache.v[at].cpu(), _encoded(dtype, v_new[row].cpu())[0])


def test_append_and_read_without_pages():
    # Rows at negative positions, without a page, of nobody; bad pages are counted, queries are rotated all the same.
    x = make_paged4([20, 2, 40], [2, 2, 3], D=128, page=16, seed=3)
    cache, batch, _ = x.device()
    x.table[0, 1], x.table[2, 2] = -1, 1 << 20
    table = x.table.to(dev())
    start = _ints([1, 3, 7, 10])                           # sequence 1: 4 rows, 2 tokens
    batch = qsa.PagedBatch(table, batch.lens, start, n_rows=11, max_rows=4)
    k_new = torch.randn(11, 2, 128, device=dev()).bfloat16()
    q, q_out = torch.randn(11, 24, 128, device=dev()).bfloat16(), torch.full((11, 24, 128), 9.0, device=dev()).bfloat16()
    before = cache.k.clone(), cache.v.clone(), cache.kv_scale.clone()
    rope = qsa.Rope(128)
    qsa.paged_append(cache, batch, k_new, k_new, rope=rope, q=q, q_out=q_out)
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "5 page table entries" in why
    pos = _ints([0, 18, 19, -2, -1, 0, 1, 37, 38, 39, 0])
    want_q = qsa.rotate(rope, pos, q.clone())
    assert torch.equal(q_out[1:10], want_q[1:10]) and (q_out[[0, 10]] == 9).all()
    want_k = qsa.rotate(rope, pos, k_new.clone()).cpu()
    for row, p in ((5, 0), (6, 1)):
        before[0][x.table[1, 0], :, p], s = (y.to(dev()) for y in _encoded("q4", want_k[row]))
        before[1][x.table[1, 0], :, p], s2 = (y.to(dev()) for y in _encoded("q4", k_new[row].cpu()))
        before[2][x.table[1, 0], :, p] = torch.cat((s, s2), -1)
    assert all(torch.equal(a, b) for a, b in zip(before, (cache.k, cache.v, cache.kv_scale)))
    k_out, v_out = (torch.full((11, 2, 128), 7.0, device=dev()) for _ in range(2))
    qsa.paged_read(cache, batch, k_out, v_out)
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "5 page table entries" in why
    keep = [0, 1, 2, 3, 4, 7, 8, 9, 10]
    assert (k_out[keep] == 7).all() and (v_out[keep] == 7).all()
    code, s, m = split4(*(y[:, None] for y in encode4(want_k[5])))
    assert torch.allclose(k_out[5].cpu().double(), (code * s + m)[:, 0], rtol=0, atol=1e-6)


def test_blocks_that_4_bits_do_not_hold():
    x = make_paged4([8], [8], D=256, page=16, seed=4)
    cache, batch, _ = x.device()
    new = torch.randn(8, 2, 256, device=dev()).bfloat16()
    new[0, 0, 5], new[1, 1, 33], new[2, 0, 70], new[3, 1, 255] = float("nan"), float("inf"), float("-inf"), 3e38
    new[3, 0, 130] = 65536.0
    new[7, 0, 0], new[7, 0, 1] = 65280.0, -65280.0
    qsa.paged_append(cache, batch, new, new)
    for i in range(8):
        c, p = encode4(new[i].float().cpu())
        at = (int(x.table[0, 0]), slice(None), i)
        assert torch.equal(cache.k[at].cpu(), c) and torch.equal(cache.v[at].cpu(), c)
        got = cache.kv_scale[at].cpu().reshape(2, 2, 8, 2)
        for w in range(2):
            assert torch.equal(torch.isnan(got[:, w, :, 0]), torch.isnan(p[..., 0]))
            ok = ~torch.isnan(p[..., 0])
            assert torch.equal(got[:, w][ok], p[ok])
    assert not torch.isnan(p[..., 0]).any()                # (the largest magnitudes that are held)
    k_out = torch.empty(8, 2, 256, device=dev())
    qsa.paged_read(cache, batch, k_out, torch.empty_like(k_out))
    bad = torch.isnan(k_out).reshape(8, 2, 8, 32)
    assert bad.all(-1).nonzero().tolist() == [[0, 0, 0], [1, 1, 1], [2, 0, 2], [3, 0, 4], [3, 1, 7]]
    assert int(bad.sum()) == 5 * 32 and qsa.check_device_status() == (0, "")


# ------------------------------------------------------------------ reading
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32", "q4"])
@pytest.mark.parametrize("D,page,order,Hkv", [(128, 16, "head", 2), (256, 64, "token", 2), (128, 1024, "token", 5), (256, 32, "head", 1)])
def test_read(dtype, D, page, order, Hkv):
    lens, rows = [1, 33, 500, 70, 64], [1, 33, 123, 0, 2]
    x, cache, batch, _ = _state(dtype, lens, rows, D=D, page=page, order=order, Hkv=Hkv, G=1, seed=5, pad_rows=2)
    n = x.q.shape[0]
    want = [torch.cat([y[:, -r:].transpose(0, 1) for y, r in ((x.seq_kv(i)[w], r) for i, r in enumerate(rows)) if r]) for w in range(2)]
    for t in (torch.float32, torch.bfloat16):
        out = [torch.full((n, Hkv, D), 7.0, dtype=t, device=dev()) for _ in range(2)]
        qsa.paged_read(cache, batch, *out)
        for got, ref in zip(out, want):
            # A product and a sum in one rounding to binary32, one to the type.
            tol = (2.0 ** -24 + (2.0 ** -8 if t is torch.bfloat16 and dtype not in ("bf16",) else 0.0)) * ref.abs() * 1.01 + 1e-40
            assert ((got[:-2].double().cpu() - ref).abs() <= tol).all() and (got[-2:] == 7).all()
    assert qsa.check_device_status() == (0, "")


def test_read_of_many_rows_and_sequences():
    # More rows than there are warps to give one each, more sequences than rows of a warp.
    lens = [1 + (i * 37) % 90 for i in range(600)]
    x = make_paged4(lens, lens, D=128, Hkv=1, G=1, page=16, seed=6)
    cache, batch, _ = x.device()
    k_out, v_out = (torch.empty(sum(lens), 1, 128, device=dev()) for _ in range(2))
    qsa.paged_read(cache, batch, k_out, v_out)
    for w, got in enumerate((k_out, v_out)):
        want = torch.cat([x.seq_kv(i)[w].transpose(0, 1) for i in range(600)])
        assert (got.double().cpu() - want).abs().max() <= 2.0 ** -23 * want.abs().max()
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("dtype", ["bf16", "q4"])
def test_append_with_rotation_replayed_and_on_another_stream(dtype):
    x, cache, batch, _ = _state(dtype, [60, 30], [2, 1], D=128, page=16, seed=7)
    k_new, q = torch.randn(3, 2, 128, device=dev()).bfloat16(), torch.randn(3, 24, 128, device=dev()).bfloat16()
    q_out, rope = torch.empty_like(q), qsa.Rope(128)
    out = [torch.empty(3, 2, 128, device=dev()) for _ in range(2)]
    call = lambda s=None: (qsa.paged_append(cache, batch, k_new, k_new, s, rope=rope, q=q, q_out=q_out),
                           qsa.paged_read(cache, batch, *out, s))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([60, 30], [33, 17], [2, 1]):
        batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for o in out:
            o.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        pos = torch.tensor([lens[0] - 2, lens[0] - 1, lens[1] - 1])
        assert_turned(q_out, q.cpu(), pos, 128, False, rope.frequencies)
        k = turned(k_new.cpu(), pos, 128, False, rope.frequencies)
        step = 0.0 if dtype == "bf16" else float((k.abs().amax() * 2 / 15))
        assert (out[0].double().cpu() - k).abs().max() <= step + 2.0 ** -7 * k.abs().max()
    assert qsa.check_device_status() == (0, "")
