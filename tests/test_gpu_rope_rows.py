"""Calls of so many rows that a CTA takes two or four of them, and of many sequences: the same bits as calls of few
rows and sequences."""
import random

import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import dev

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


def rows_of(times, more):
    """Rows just above those that leave `times` CTAs of one, two ... rows for every SM."""
    return times * torch.cuda.get_device_properties(0).multi_processor_count + more


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("heads,D,rot,times,more", [(3, 128, 128, 8, 1), (24, 256, 64, 8, 3), (5, 128, 48, 16, 1), (24, 128, 128, 16, 2),
                                                    (1, 16, 16, 16, 3), (7, 1024, 256, 32, 7), (2, 256, 256, 32, 5)])
def test_rotations_of_many_rows(dtype, pairs, heads, D, rot, times, more):
    n = rows_of(times, more)
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, heads, D, device=dev(), generator=g).to(dtype)
    pos = torch.randint(-1000, 2 ** 31 - 1, (n,), generator=g, device=dev(), dtype=torch.int32)
    r = qsa.Rope(rot, base=1e5, pairs=pairs)
    want = torch.cat([qsa.rotate(r, p.contiguous(), y.contiguous(), torch.empty_like(y)) for p, y in zip(pos.split(100), x.split(100))])
    room = torch.full((n + 4, heads, D), 7.0, device=dev(), dtype=dtype)
    qsa.rotate(r, pos, x, room[2:n + 2])
    assert torch.equal(room[2:n + 2], want) and (room[:2] == 7).all() and (room[n + 2:] == 7).all()
    room[2:n + 2] = x                                      # in place
    qsa.rotate(r, pos, room[2:n + 2])
    assert torch.equal(room[2:n + 2], want) and (room[:2] == 7).all() and (room[n + 2:] == 7).all()


def many(n_seqs, n, rng):
    """(lens, rows) of n_seqs sequences with n rows: some have none, a few have many."""
    rows = [0] * n_seqs
    for i in (0, n_seqs // 2, n_seqs - 2):
        rows[i] = n // 5
    left = n - sum(rows)
    while left:
        i = rng.randrange(n_seqs)
        if i % 7 and i != n_seqs - 1:
            rows[i] += 1
            left -= 1
    return [max(r, 1) + rng.randint(0, 60) for r in rows], rows


def caches(kind, lens, Hkv, D, page, rng):
    counts = [-(-m // page) for m in lens]
    ids = list(range(sum(counts) + 2))
    rng.shuffle(ids)
    table, at = torch.full((len(lens), max(counts) + 1), -1, dtype=torch.int32), 0
    for i, c in enumerate(counts):
        table[i, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
        at += c
    return [qsa.PagedCache.zeros(len(ids), Hkv, page, D, kind) for _ in range(2)], table


def held(c):
    return [t.view(torch.uint8) for t in (c.k, c.v)] + ([] if c.kv_scale is None else [c.kv_scale.view(torch.int16)])


@pytest.mark.parametrize("kind", [qsa.BF16, qsa.F32, qsa.FP8, qsa.Q4], ids=["bf16", "f32", "fp8", "q4"])
@pytest.mark.parametrize("D,pairs,n_seqs,times,more", [(128, False, 33, 8, 1), (256, True, 64, 8, 3), (128, True, 288, 16, 1),
                                                       (256, False, 289, 16, 3), (128, False, 600, 16, 2), (256, True, 32, 16, 1),
                                                       (128, True, 545, 1, 3), (256, False, 40, 0, 60)])
def test_appends_of_many_rows_and_sequences(kind, D, pairs, n_seqs, times, more):
    rng = random.Random(n_seqs)
    before, after, Hkv, G, page = 3, 2, 2, 3, 16
    n = rows_of(times, more) if times else more            # of sequences; rows of nobody lie on both sides
    lens, rows = many(n_seqs, n, rng)
    (cache, plain), table = caches(kind, lens, Hkv, D, page, rng)
    starts = [before]
    for r in rows:
        starts.append(starts[-1] + r)
    total = starts[-1] + after
    g = torch.Generator(device="cuda").manual_seed(n)
    fused = torch.randn(total, Hkv * (G + 2), D, device=dev(), generator=g).to(cache.row_dtype)
    q, k_new, v_new = fused[:, :Hkv * G], fused[:, Hkv * G:Hkv * (G + 1)], fused[:, Hkv * (G + 1):]
    rope = qsa.Rope(D if pairs else 64, base=1e4, pairs=pairs)
    batch = qsa.PagedBatch(table.to(dev()), _ints(lens), _ints(starts), n_rows=total, max_rows=max(rows))
    q_out = torch.full((total, Hkv * G, D), 9.0, device=dev()).to(cache.row_dtype)
    q_few = q_out.clone()
    qsa.paged_append(cache, batch, k_new, v_new, rope=rope, q=q, q_out=q_out)
    # The same, a sequence and at most 100 rows a call.
    for i, r in enumerate(rows):
        for j in range(0, r, 100):
            m, at = min(100, r - j), starts[i] + j
            part = qsa.PagedBatch(batch.table[i:i + 1], _ints([lens[i] - r + j + m]), _ints([0, m]), n_rows=m)
            s = slice(at, at + m)
            qsa.paged_append(plain, part, k_new[s], v_new[s], rope=rope, q=q[s], q_out=q_few[s])
    for a, b in zip(held(cache), held(plain)):
        assert torch.equal(a, b)
    assert torch.equal(q_out, q_few) and (q_out[:before] == 9).all() and (q_out[total - after:] == 9).all()
    # Without a rotation, and read back.
    qsa.paged_append(cache, batch, v_new, k_new)
    for i, r in enumerate(rows):
        for j in range(0, r, 100):
            m, at = min(100, r - j), starts[i] + j
            part = qsa.PagedBatch(batch.table[i:i + 1], _ints([lens[i] - r + j + m]), _ints([0, m]), n_rows=m)
            qsa.paged_append(plain, part, v_new[at:at + m], k_new[at:at + m])
    for a, b in zip(held(cache), held(plain)):
        assert torch.equal(a, b)
    back, few = ([torch.full((total, Hkv, D), 5.0, device=dev()) for _ in range(2)] for _ in range(2))
    qsa.paged_read(cache, batch, *back)
    for i, r in enumerate(rows):
        if r:
            part = qsa.PagedBatch(batch.table[i:i + 1], batch.lens[i:i + 1], _ints([0, r]), n_rows=r)
            qsa.paged_read(plain, part, *(t[starts[i]:starts[i + 1]] for t in few))
    assert all(torch.equal(a, b) for a, b in zip(back, few))
    assert qsa.check_device_status() == (0, "")


@pytest.mark.parametrize("kind", [qsa.BF16, qsa.F32, qsa.FP8, qsa.Q4], ids=["bf16", "f32", "fp8", "q4"])
@pytest.mark.parametrize("D,times,more", [(128, 64, 3), (256, 128, 5), (256, 256, 1)])
def test_reads_of_many_rows(kind, D, times, more):
    # Two, four and eight rows a warp, several sequences in one.
    rng = random.Random(times)
    n, Hkv, page = rows_of(times, more), 1, 64
    lens, rows = many(50, n, rng)
    (cache, _), table = caches(kind, lens, Hkv, D, page, rng)
    g = torch.Generator(device="cuda").manual_seed(n)
    for t in (cache.k, cache.v):
        if kind in (qsa.FP8, qsa.Q4):
            t.view(torch.uint8).copy_(torch.randint(0, 120, t.shape, generator=g, device=dev(), dtype=torch.uint8))
        else:
            t.copy_(torch.randn(t.shape, generator=g, device=dev()))
    if cache.kv_scale is not None:
        cache.kv_scale.copy_(torch.randn(cache.kv_scale.shape, generator=g, device=dev()))
    starts = [1]
    for r in rows:
        starts.append(starts[-1] + r)
    total = starts[-1] + 3
    batch = qsa.PagedBatch(table.to(dev()), _ints(lens), _ints(starts), n_rows=total, max_rows=max(rows))
    for t in (torch.float32, torch.bfloat16):
        back, few = ([torch.full((total, Hkv, D), 5.0, device=dev(), dtype=t) for _ in range(2)] for _ in range(2))
        qsa.paged_read(cache, batch, *back)
        for i, r in enumerate(rows):
            for j in range(0, r, 2000):
                m = min(2000, r - j)
                part = qsa.PagedBatch(batch.table[i:i + 1], _ints([lens[i] - r + j + m]), _ints([0, m]), n_rows=m)
                qsa.paged_read(cache, part, *(y[starts[i] + j:starts[i] + j + m] for y in few))
        assert all(torch.equal(a, b) for a, b in zip(back, few))
    assert qsa.check_device_status() == (0, "")
