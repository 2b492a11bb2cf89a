"""Calls over selected pages that the documentation allows and that sit at its edges: slots named twice, empty
batches, sound sequences beside malformed ones, the kernels for runs of tokens on two streams and again and again."""
import numpy as np
import pytest

from paged_kv_cache_201_gb300 import workloads as W
from tests import _gpu
from tests import _sparse_ref as R
from tests.test_serving_step_gpu import _append_case, _check_append, _lists, _raw, _run_append, _shares, _t, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,ps,seq", [("bf16", 128, 16, 40), ("f32", 64, 32, 50), ("f16", 256, 64, 130),
                                            ("bf16", 64, 64, 2200)])
def test_append_slot_named_twice(pa, dtype, D, ps, seq):  # noqa: F811
    """The slot holds either token's elements; no envelope could bound both, so the page has none.  Every other
    page is as without it (seq 2200: several tokens a warp)."""
    b, slots, kn, vn = _append_case(D + ps, [seq], [seq], 8, D, ps, dtype, pads=2)
    pages = slots[:seq] // ps
    first = np.flatnonzero(pages == pages[ps + 3])  # the second page's tokens
    slots[first[5]] = slots[first[2]]   # its row 5 is not written, its row 2 twice
    slots[first[-1]] = slots[first[-3]]  # its last row neither
    k, v = b.k.copy(), b.v.copy()
    e, s = np.full((b.P, 8, 2, D), 77, np.int8), np.full((b.P, 8), -1.0, np.float32)
    R.append(kn, vn, slots, k, v, dtype, e, s)
    page = pages[ps + 3]
    e[page], s[page] = 0, np.inf
    gk, gv, ge, gs = _run_append(pa, b, slots, kn, vn)
    np.testing.assert_array_equal(gs, s)
    np.testing.assert_array_equal(ge, e)
    for t1, t2 in ((first[2], first[5]), (first[-3], first[-1])):
        row = slots[t1] % ps
        for got, new, want in ((gk, kn, k), (gv, vn, v)):
            assert ((got[page, row] == new[t1]) | (got[page, row] == new[t2])).all()
            want[page, row] = got[page, row]
    np.testing.assert_array_equal(_raw(gk), _raw(k))
    np.testing.assert_array_equal(_raw(gv), _raw(v))
    assert pa.paged_attn_last_error_word() == 0


@pytest.mark.parametrize("other_stream", [False, True])
def test_step_tables_of_an_empty_batch(pa, other_stream):  # noqa: F811
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    none, free = torch.zeros(0, **i32), torch.arange(9, **i32)
    got = pa.step_tables(none, none, free, torch.tensor([5], **i32), torch.zeros((0, 4), **i32), 6, 16, 9,
                         stream=torch.cuda.Stream() if other_stream else None)
    torch.cuda.synchronize()
    assert [x.tolist() for x in got] == [[], [], [0], [-1] * 6, [5]]
