"""Scratch that a call allocates itself belongs to the stream the call runs on."""
import pytest
import torch

import indexed_sparse_attention_gb300 as qsa
from indexed_sparse_attention_gb300 import paged
from paged_cases import dev, make_paged


@pytest.fixture
def allocations(monkeypatch):
    """Without a GPU: the stream that is the current one at each allocation of scratch."""
    current, seen, empty = ["the current stream"], [], torch.empty

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *_):
            current.pop()

    def fake_empty(*size, **kw):
        if kw.get("dtype") is torch.uint8:
            seen.append(current[-1])
            kw.pop("device", None)
        return empty(*size, **kw)

    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: f"stream {handle} of {device}")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: f"default stream of {device}")
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", fake_empty)
    yield seen
    assert len(current) == 1


def test_scratch_is_allocated_on_the_stream_of_the_call(allocations):
    assert paged._scratch(100, torch.device("cuda", 0), None).numel() == 100
    assert paged._scratch(0, torch.device("cuda", 0), 77).numel() == 16
    paged._scratch(9, torch.device("cuda", 0), 0)           # the handle of the default stream
    assert allocations == ["the current stream", "stream 77 of cuda:0", "default stream of cuda:0"]


def test_scratch_of_the_layer_step_calls_too(allocations, monkeypatch):
    # Every call of the package that allocates its scratch when none is given, over a library that only says "64 bytes".
    class Fake:
        def __getattr__(self, name):
            return lambda *args: 64 if name.endswith("workspace_size") else 0

    monkeypatch.setattr(qsa, "lib", lambda: Fake())
    z = torch.zeros
    pooled, scores, q_idx = z(16, 128), z(1, 16), z(1, 4, 128)
    sel, cnt, q, out = z(1, 16, dtype=torch.int32), z(1, dtype=torch.int32), z(1, 4, 128), z(1, 4, 128)
    seq = qsa.Seq(40, 1, pooled, [qsa.Segment(z(2, 40, 128), z(2, 40, 128), 0)], idx_keys=z(40, 128))
    calls = [lambda s: qsa.score_blocks([seq], q_idx, scores, s),
             lambda s: qsa.pool_score_blocks([seq], q_idx, scores, s),
             lambda s: qsa.select_topk([seq], scores, sel, cnt, stream=s),
             lambda s: qsa.score_select_topk([seq], q_idx, scores, sel, cnt, stream=s),
             lambda s: qsa.score_select_topk_blocked([seq], q_idx, sel, cnt, stream=s),
             lambda s: qsa.append_score_blocks(seq, z(2, 1, 128), z(2, 1, 128), z(1, 128), q_idx, scores, s),
             lambda s: qsa.sparse_attn([seq], q, sel, cnt, out, stream=s)]
    for call in calls:
        allocations.clear()
        call(77)
        assert allocations == ["stream 77 of cpu"]


@pytest.mark.gpu
def test_the_handle_of_the_default_stream():
    # Scratch of a call with handle 0 is the default stream's, whichever is the current one.
    seen = {}
    side = torch.cuda.Stream()
    for name, stream in (("default", torch.cuda.default_stream()), ("handle", 0)):
        with torch.cuda.stream(side):
            ws = paged._scratch(40 << 20, dev(), stream)
            seen[name] = ws.data_ptr()
            del ws
    # (The block went back to the stream it came from and is handed out there again.)
    ws = torch.empty(40 << 20, dtype=torch.uint8, device=dev())
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert seen["handle"] == seen["default"] == ws.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_calls_without_a_workspace_on_streams_that_run_at_once(handle):
    # Long calls on the current stream whose scratch is free for Python while they still run, and a call
    # on a stream that nothing orders behind them.
    long = make_paged([9000, 3000], [600, 1], dtype="bf16", D=128, page=64, seed=70)
    short = make_paged([4000, 50], [3, 1], dtype="bf16", D=128, page=64, seed=71)
    side = torch.cuda.Stream()
    cases = []
    for x in (long, short):
        cache, batch, q = x.device()
        # (One shape of call, so that one's scratch would fit the other.)
        batch = qsa.PagedBatch(batch.table, batch.lens, batch.row_start, n_rows=batch.n_rows, max_rows=600)
        out, lse = torch.empty(q.shape, device=dev()), torch.empty(q.shape[:2], device=dev())
        qsa.paged_attn(cache, batch, q, out, lse)
        torch.cuda.synchronize()
        cases.append((cache, batch, q, out, lse, out.clone(), lse.clone()))
    (lc, lb, lq, lo, ll, want_lo, want_ll), (sc, sb, sq, so, sl, want_so, want_sl) = cases
    for _ in range(20):
        lo.zero_()
        so.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            qsa.paged_attn(lc, lb, lq, lo, ll)
        for _ in range(3):
            qsa.paged_attn(sc, sb, sq, so, sl, stream=side.cuda_stream if handle else side)
        filler = torch.full((1 << 22,), 3.0, device=dev())       # may not take the side stream's scratch either
        torch.cuda.synchronize()
        assert torch.equal(lo, want_lo) and torch.equal(ll, want_ll)
        assert torch.equal(so, want_so) and torch.equal(sl, want_sl)
        del filler
    assert qsa.check_device_status() == (0, "")
