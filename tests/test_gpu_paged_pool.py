"""The keeping of pages at its ends: pools that run out inside a serving step,
requests for more pages than 32 bits count, tables that name pages nobody counts, and
lengths below zero."""
import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from paged_cases import Paged, assert_attended, attend64, dev

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


# ------------------------------------------------------------------ extend that is not served
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_a_step_whose_extend_is_not_served_leaves_the_tokens(dtype):
    P, D = 16, 128
    kind = {"bf16": torch.bfloat16, "fp8": torch.uint8, "f32": torch.float32}[dtype]
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    k, v = (torch.zeros(4, 2, P, D, dtype=kind, device=dev()) for _ in range(2))
    sc = torch.zeros(4, 2, P, 2, dtype=torch.float16, device=dev()) if dtype == "fp8" else None
    cache = qsa.PagedCache(k, v, sc)
    pool = qsa.PagePool.empty(3, 4, [cache])
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda n, h: torch.randn(n, h, D, generator=g, device=dev()).to(act)

    def step(who, counts, rows):
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        pool.extend(_ints(who), _ints(counts))
        batch = qsa.PagedBatch(pool.table, pool.step_lens, _ints(starts), n_rows=starts[-1], max_rows=max(rows))
        st = qsa.PagedStep(cache, batch, rand(starts[-1], 4))
        st.run(rand(starts[-1], 2), rand(starts[-1], 2))
        torch.cuda.synchronize()
        return st

    step([0], [2 * P], [2 * P, 0, 0])                     # two full pages ...
    pool.fork(_ints([0]), _ints([1]))                     # ... shared with place 1
    step([2], [P + 3], [0, 0, P + 3])                     # the other two, the last one with room
    assert qsa.check_device_status() == (0, "")
    kept = [t.clone() for t in (k, v)] + [pool.table.clone(), pool.lens.clone(), pool.refs.clone()]
    # Places 0 and 1 find no page; place 2 has room in its last one.
    st = step([0, 2, 1], [1, 2, 3], [1, 3, 2])
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK
    assert pool.lens.tolist() == [2 * P, 2 * P, P + 5] and pool.step_lens.tolist() == [0, 0, P + 5]
    last, at = int(pool.table[2, 1]), slice(3, 5)
    for now, was in zip((k, v), kept):
        assert not torch.equal(now[last, :, at], was[last, :, at])
        was[last, :, at] = now[last, :, at]
        assert torch.equal(now, was)                      # every other token is as it was
    assert torch.equal(pool.table, kept[2]) and torch.equal(pool.refs, kept[4])
    assert (st.out[:4] == 0).all() and torch.isneginf(st.lse[:4]).all()
    assert torch.isfinite(st.lse[4:]).all() and (st.out[4:] != 0).any()
    assert qsa.check_device_status() == (0, "")
    # With a page given back, the next step is an ordinary one again.
    pool.free(_ints([2]))
    st = step([0], [1], [1, 0, 0])
    assert pool.step_lens.tolist() == [2 * P + 1, 2 * P, 0] and torch.isfinite(st.lse).all()
    assert qsa.check_device_status() == (0, "")


def test_step_lengths_of_refused_requests():
    # Repeated places, places outside, lengths below zero and behind the table; more places than threads.
    places = 3000
    pool = qsa.PagePool(torch.full((places, 2), -1, dtype=torch.int32, device=dev()), _ints([0] * places),
                        _ints([0] * 64), page_tokens=16)
    pool.extend(_ints([5, 7, 5, -1, places, 9, 2999, 11]), _ints([4, 20, 1, 1, 1, -1, 32, 33]))
    want = {7: 20, 2999: 32}
    lens = {5: 4, **want}
    assert {i: n for i, n in enumerate(pool.lens.tolist()) if n} == lens
    assert {i: n for i, n in enumerate(pool.step_lens.tolist()) if n} == want
    pool.extend(_ints([9]), _ints([3]))                   # what was refused before is over
    assert {i: n for i, n in enumerate(pool.step_lens.tolist()) if n} == {**lens, 9: 3}
    pool.free(_ints([7]))
    pool.extend(_ints([]), _ints([]))                     # no request: the pool's lengths
    assert torch.equal(pool.step_lens, pool.lens)
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


def test_captured_steps_until_the_pool_is_full():
    # One captured step (extend, append, attend) replayed past the end of the pool: the rows that found room are
    # kept, and each replay's attention is that of the tokens there are.
    P, D, n_pages, steps = 16, 128, 5, 60
    k, v = (torch.zeros(n_pages, 2, P, D, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    pool = qsa.PagePool.empty(2, 4, [qsa.PagedCache(k, v)])
    who, one, start = _ints([0, 1]), _ints([1, 1]), _ints([0, 1, 2])
    batch = qsa.PagedBatch(pool.table, pool.step_lens, start, n_rows=2, max_rows=1)
    q = torch.randn(2, 4, D, generator=torch.Generator().manual_seed(2)).bfloat16()
    st = qsa.PagedStep(pool.caches[0], batch, q.to(dev()))
    rows = torch.randn(steps, 2, 2, 2, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    new = torch.zeros(2, 2, 2, D, dtype=torch.bfloat16, device=dev())      # [K or V, sequence, head, channel]
    pool.extend(who, _ints([0, 0]))
    st.run(new[0], new[1])                                # (once before the capture; no tokens yet)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pool.extend(who, one)
        st.run(new[0], new[1])
    tokens = [[], []]
    for i in range(steps):
        new.copy_(rows[i])
        graph.replay()
        torch.cuda.synchronize()
        lens = pool.step_lens.tolist()
        for s in (0, 1):
            if lens[s]:
                tokens[s].append(rows[i][:, s])
            else:
                assert (st.out[s] == 0).all() and torch.isneginf(st.lse[s]).all()
        assert pool.lens.tolist() == [len(t) for t in tokens]
    assert [len(t) for t in tokens] == [3 * P, 2 * P]     # five pages, the first request's place first
    n = max(len(t) for t in tokens)
    plain = Paged(torch.zeros(2, 2, n, D), torch.zeros(2, 2, n, D), None, torch.arange(2, dtype=torch.int32)[:, None],
                  [len(t) for t in tokens], [1, 1], torch.tensor([0, 1, 2]), q, n, "head")
    for s in (0, 1):
        for t, row in enumerate(tokens[s]):
            plain.k[s, :, t], plain.v[s, :, t] = row[0].float(), row[1].float()
    batch = qsa.PagedBatch(pool.table, pool.lens, start, n_rows=2, max_rows=1)
    out, lse = torch.empty(2, 4, D, device=dev()), torch.empty(2, 4, device=dev())
    qsa.paged_attn(pool.caches[0], batch, q.to(dev()), out, lse)
    assert_attended(out, lse, attend64(plain))
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


# ------------------------------------------------------------------ requests of any size
def test_requests_for_more_pages_than_32_bits_count():
    # 140 places that want 2^24 pages each: 2.3e9, of which the pool has 100.
    ld, places, n_pages = 1 << 24, 143, 100
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 10 GB")
    table = torch.full((places, ld), -1, dtype=torch.int32, device=dev())
    pool = qsa.PagePool(table, _ints([0] * places), _ints([0] * n_pages), page_tokens=16)
    pool.extend(_ints(list(range(places))), _ints([33] + [1 << 28] * 140 + [16, 0]))
    assert pool.lens.tolist() == [33] + [0] * (places - 1)      # (the others are behind requests that take all)
    assert pool.step_lens.tolist() == pool.lens.tolist()
    assert table[0, :3].tolist() == [0, 1, 2] and pool.refs.tolist() == [1] * 3 + [0] * (n_pages - 3)
    assert int((table.view(-1)[3:] != -1).sum()) == 0
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "141 page requests" in why
    pool.extend(_ints([1, 142]), _ints([16 * 97, 5]))           # all that is left, then one more
    assert pool.lens.tolist() == [33, 16 * 97] + [0] * (places - 2)
    assert table[1, :97].tolist() == list(range(3, 100))
    assert qsa.check_device_status()[0] == qsa.ERR_DEVICE_CHECK


# ------------------------------------------------------------------ compact
def test_compact_keeps_entries_of_pages_that_nobody_counts():
    k, v = (torch.randn(12, 2, 16, 128, device=dev()).bfloat16() for _ in range(2))
    pool = qsa.PagePool.empty(3, 4, [qsa.PagedCache(k, v)])
    pool.table.copy_(torch.tensor([[9, 3, -1, -1], [10, 11, 40, -1], [-1] * 4], dtype=torch.int32))
    pool.lens.copy_(torch.tensor([20, 40, 0], dtype=torch.int32))
    pool.refs[9] = pool.refs[3] = pool.refs[11] = 1             # nobody counts page 10, and page 40 does not exist
    was = k.clone()
    for junk in (0x5A, 0xFF, 0x00):                             # (whatever the workspace held before)
        pool.ws.fill_(junk)
        pool.compact()
        assert pool.table.tolist() == [[1, 0, -1, -1], [10, 2, 40, -1], [-1] * 4]      # pages 3, 9 and 11 to 0, 1 and 2
        assert pool.refs.tolist() == [1] * 3 + [0] * 9
        assert all(torch.equal(k[to], was[page]) for to, page in ((0, 3), (1, 9), (2, 11)))


# ------------------------------------------------------------------ copy
def test_copy_in_caches_of_unequal_numbers_of_pages():
    # A pool has the pages that all of its caches have; 35 of them take two launches.
    n = [8, 6] + [7] * 33
    caches = [qsa.PagedCache(*(torch.randn(m, 2, 16, 128, device=dev()).bfloat16() for _ in range(2))) for m in n]
    pool = qsa.PagePool.empty(2, 2, caches)
    assert pool.refs.numel() == 6
    want = [(c.k.clone(), c.v.clone()) for c in caches]
    pool.copy(_ints([1, 6, 5]), _ints([2, 3, 7]))               # pages 6 and 7 are not in every cache
    for c, (k, v) in zip(caches, want):
        k[2], v[2] = k[1], v[1]
        assert torch.equal(c.k, k) and torch.equal(c.v, v)
    status, why = qsa.check_device_status()
    assert status == qsa.ERR_DEVICE_CHECK and "page requests" in why


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("length", [0, -1, -(2 ** 31), -(2 ** 31) + 2])
def test_append_to_sequences_of_no_tokens(length):
    # The rows sit before the first token and are skipped without a report, as attention gives them nothing.
    # (The table has a page for each position that fits 31 bits.)
    page, ld = 1024, 1 << 21
    k, v = (torch.zeros(2, 1, page, 128, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    table = torch.zeros(1, ld, dtype=torch.int32, device=dev())
    cache, batch = qsa.PagedCache(k, v), qsa.PagedBatch(table, _ints([length]), _ints([0, 5]), n_rows=5)
    rows = torch.ones(5, 1, 128, dtype=torch.bfloat16, device=dev())
    qsa.paged_append(cache, batch, rows, rows)
    out, lse = torch.ones(5, 4, 128, device=dev()), torch.ones(5, 4, device=dev())
    qsa.paged_attn(cache, batch, torch.ones(5, 4, 128, dtype=torch.bfloat16, device=dev()), out, lse)
    assert not k.any() and not v.any() and not out.any() and torch.isneginf(lse).all()
    assert qsa.check_device_status() == (0, "")
