"""Tensors on another device than the rest of a call, where neither is a GPU (CPU and meta tensors have the same
device number): the refusal names them."""
import pytest
import torch

import indexed_sparse_attention_gb300 as qsa


def i32(*s, **kw):
    return torch.zeros(*s, dtype=torch.int32, **kw)


def bf16(*s, **kw):
    return torch.zeros(*s, dtype=torch.bfloat16, **kw)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from indexed_sparse_attention_gb300 import build
    build.build()


def test_rows_and_batches_of_another_device_than_the_cache():
    cache = qsa.PagedCache(bf16(4, 2, 16, 128), bf16(4, 2, 16, 128))
    batch = qsa.PagedBatch(i32(2, 4), i32(2), i32(3), n_rows=2)
    far = qsa.PagedBatch(i32(2, 4, device="meta"), i32(2, device="meta"), i32(3, device="meta"), n_rows=2)
    q, new, lse, rope = bf16(2, 24, 128), bf16(2, 2, 128), torch.zeros(2, 24), qsa.Rope(64)
    q_far, new_far, lse_far = (t.to("meta") for t in (q, new, lse))
    for call, what in ((lambda: qsa.paged_attn(cache, batch, q_far, q.clone()), "q must be"),
                       (lambda: qsa.paged_attn(cache, batch, q, q_far), "out must be"),
                       (lambda: qsa.paged_attn(cache, batch, q, q.clone(), lse_far), "lse must be"),
                       (lambda: qsa.paged_append(cache, batch, new_far, new), "k_new must be"),
                       (lambda: qsa.paged_append(cache, batch, new, new_far), "v_new must be"),
                       (lambda: qsa.paged_append(cache, batch, new, new, rope=rope, q=q_far, q_out=q), "q must be"),
                       (lambda: qsa.paged_append(cache, batch, new, new, rope=rope, q=q, q_out=q_far), "q_out must be"),
                       (lambda: qsa.paged_read(cache, batch, new_far, new), "k_out must be"),
                       (lambda: qsa.paged_read(cache, batch, new, new_far), "v_out must be"),
                       (lambda: qsa.paged_attn(cache, far, q, q.clone()), "another device"),
                       (lambda: qsa.paged_append(cache, far, new, new), "another device"),
                       (lambda: qsa.paged_read(cache, far, new, new.clone()), "another device"),
                       (lambda: qsa.PagedStep(cache, batch, q_far), "q must be"),
                       (lambda: qsa.PagedStep(cache, batch, q_far, rope=rope), "q must be")):
        with pytest.raises(ValueError, match=what):
            call()


def test_rotations_of_tensors_on_two_devices():
    rope, x, pos = qsa.Rope(64), bf16(2, 24, 128), i32(2)
    with pytest.raises(ValueError, match="one shape, dtype and device"):
        qsa.rotate(rope, pos, x, x.to("meta"))
    with pytest.raises(ValueError, match="positions is on meta"):
        qsa.rotate(rope, pos.to("meta"), x)
    with pytest.raises(ValueError, match="not on a GPU"):
        qsa.rotate(rope, pos.to("meta"), x.to("meta"))
