"""A step with a rope attends with the queries that its append has rotated: not before it."""
import pytest
import torch

import indexed_sparse_attention_gb300 as qsa


def i32(*s, **kw):
    return torch.zeros(*s, dtype=torch.int32, **kw)


def a_step(device, **kw):
    cache = qsa.PagedCache.zeros(4, 2, 16, 128, qsa.Q4, device=device)
    batch = qsa.PagedBatch(i32(2, 4, device=device), i32(2, device=device) + 3, torch.tensor([0, 1, 2], dtype=torch.int32, device=device),
                           n_rows=2, max_rows=1)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, h, 128, generator=g).bfloat16().to(device) for h in (24, 2, 2))
    return qsa.PagedStep(cache, batch, q, **kw), k, v


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()


def test_attend_before_the_first_append_is_refused():
    step, k, v = a_step("cpu", rope=qsa.Rope(64))
    with pytest.raises(ValueError, match="append"):
        step.attend()
    with pytest.raises(ValueError, match="not on a GPU"):
        step.run(k, v)                                     # an append that did not happen
    with pytest.raises(ValueError, match="append"):
        step.attend()
    step, _, _ = a_step("cpu")                             # without a rope there is nothing to wait for
    with pytest.raises(ValueError, match="not on a GPU"):
        step.attend()


@pytest.mark.gpu
def test_attend_after_an_append_goes_on():
    step, k, v = a_step("cuda", rope=qsa.Rope(64))
    with pytest.raises(ValueError, match="append"):
        step.attend()
    step.append(k, v)
    first = step.attend()[0].clone()
    assert torch.isfinite(first).all() and torch.equal(step.attend()[0], first)
    step.q_in.mul_(0.5)                                    # other queries: an append takes them
    assert torch.equal(step.attend()[0], first)
    assert not torch.equal(step.run(k, v)[0], first)
    assert qsa.check_device_status() == (0, "")
