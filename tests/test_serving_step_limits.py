"""Calls over selected pages at the edge of what they are for: refused, or with every output defined (CPU only)."""
import math

import pytest

import paged_kv_cache_201_gb300 as pa
from tests.test_serving_step_abi import FakeCuda, fake_device, lib  # noqa: F401


@pytest.mark.parametrize("scale", [-0.1, -1e-30, -math.inf, math.nan])
def test_attention_sparse_refuses_a_negative_scale(lib, fake_device, scale):  # noqa: F811
    """The selection takes the pages of largest q.k; with a negative scale those are the ones of least weight."""
    import torch
    bf, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    pool = FakeCuda(9, 16, 2, 128, dtype=bf)
    with pytest.raises(ValueError, match="scale"):
        pa.attention_sparse(FakeCuda(3, 1, 8, 128, dtype=bf), pool, pool, FakeCuda(9, 2, 2, 128, dtype=i8),
                            FakeCuda(9, 2, dtype=f32), FakeCuda(3, 6), FakeCuda(3), top_k=4, scale=scale)


@pytest.mark.parametrize("count,left", [(5, 5), (0, 0), (12, 9), (-3, 0)])
def test_step_tables_of_an_empty_batch(lib, monkeypatch, count, left):  # noqa: F811
    """No request: no slots, no query rows, and the free pages as they were.  The library has nothing to launch
    then, so host tensors do (filled with garbage before)."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(pa, "_stream", lambda s: None)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, **kw).fill_(77))
    i32 = dict(dtype=torch.int32)
    none, free = torch.zeros(0, **i32), torch.arange(9, **i32)
    lens, q_offset, q_start, slots, free_left = pa.step_tables(none, none, free, torch.tensor([count], **i32),
                                                               torch.zeros((0, 4), **i32), 6, 16, 9)
    assert lens.shape == q_offset.shape == (0,)
    assert q_start.tolist() == [0] and slots.tolist() == [-1] * 6 and free_left.tolist() == [left]
