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
