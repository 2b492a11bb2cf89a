"""Frees by clusters of CTAs where CTAs start late or go through several rounds, against sequential lists
(tests/_kv4_ref.py).  Everything is a whole number and must match exactly."""
import numpy as np
import pytest

from tests import _kv4_ref as R
from tests.test_pages_gpu import _full, _state, _t, pa  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,width", [(60, 40), (300, 40), (900, 90)])
def test_free_beside_other_work(pa, B, width):
    """Four to sixteen CTAs of a cluster, set up while the multiprocessors are taken, again and again."""
    import torch
    s = _state(B + width, B, width, 16, empty=0.05, shared=0.8)
    rows = s["rng"].permutation(B)
    want = R.free(list(rows), s["table"], s["lens"], s["shares"], s["stack"], s["count"], 16, s["P"])
    want = [_t(want[k]) for k in ("lens", "shares", "stack")] + [_t([want["left"]])]
    rows, table, lens, count = _t(rows), _t(s["table"]), _t(s["lens"]), _t([s["count"]])
    shares0, stack0 = _t(s["shares"]), _t(s["stack"])
    other, x = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda").bfloat16()
    torch.cuda.synchronize()
    wrong = _full(1, 0)
    for _ in range(100):
        with torch.cuda.stream(other):
            for _ in range(3):
                torch.mm(x, x)
        shares, stack = shares0.clone(), stack0.clone()
        lens_out, left = _full(B), _full(1)
        pa.paged_attn_free(rows, table, lens, lens_out, shares, stack, count, left, 16)
        for got, w in zip((lens_out, shares, stack, left), want):
            wrong += (got != w).any()
    assert int(wrong) == 0
    assert pa.paged_attn_last_error_word() == 0
