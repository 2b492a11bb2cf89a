"""Forks and compactions over lists of pools: a list that the copy would refuse is refused before the tables change, and a
list may be of any length."""
import numpy as np
import pytest

import paged_kv_cache_201_gb300 as pa
from paged_kv_cache_201_gb300 import build
from tests.test_serving_step_abi import FakeCuda


def _bad(make):
    """(pools, what is wrong with them): nine pages, as page_shares has."""
    import torch
    good = make(9, 4)
    yield [good, make(8, 4)], "fewer pages than counts"
    yield [make(10, 4), make(10, 4)], "more"
    yield [good, make(9)], "no page contents"
    yield [make(9, 4, strides=(8, 1))], "not dense"
    yield [good, make(9, 6, dtype=torch.uint8)], "six bytes a page"
    yield [make(9, 0)], "none"
    yield [good] * 200 + [make(9, 3, dtype=torch.uint8)], "far back in a long list"


# ----------------------------------------------------------------------------- on the host
@pytest.fixture
def calls(monkeypatch):
    import torch
    build.build()
    pa.load_library()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(pa, "_made", lambda stream, device, *wanted: [FakeCuda(1) for _ in wanted])
    made = []
    for name in ("paged_attn_fork", "paged_attn_compact"):
        monkeypatch.setattr(pa, name, lambda *a, name=name: made.append(name))
    monkeypatch.setattr(pa, "paged_attn_copy_pages", lambda pools, *a: made.append(len(pools)))
    return made


def _fork(pools, P=9):
    return pa.fork_sequences(FakeCuda(3), FakeCuda(3), FakeCuda(4, 6), FakeCuda(4), FakeCuda(P), FakeCuda(9), FakeCuda(1),
                             pools, 16)


def _compact(pools, P=9):
    return pa.compact_pages(FakeCuda(4, 6), FakeCuda(4), FakeCuda(P), FakeCuda(9), FakeCuda(1), pools, 16)


@pytest.mark.parametrize("fn", [_fork, _compact])
def test_refused_before_anything_changes(calls, fn):
    for pools, what in list(_bad(FakeCuda)) + [([FakeCuda(9, 4, device=1)], "another device"),
                                               ([FakeCuda(9, 1 << 29)], "pages of 2 GB")]:
        with pytest.raises(ValueError, match="pools"):
            fn(pools)
        assert calls == [], what


@pytest.mark.parametrize("fn,name", [(_fork, "paged_attn_fork"), (_compact, "paged_attn_compact")])
def test_lists_of_any_length(calls, fn, name):
    for n, groups in ((0, []), (1, [1]), (192, [192]), (193, [192, 1]), (500, [192, 192, 116])):
        fn(iter([FakeCuda(9, 4)] * n))
        assert calls == [name] + groups
        calls.clear()


# ----------------------------------------------------------------------------- on the GPU
def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


@pytest.mark.gpu
def test_refused_calls_leave_the_tables():
    import torch
    pa.load_library(build_if_missing=True)

    def make(*shape, dtype=torch.int32, strides=None):
        return torch.empty_strided(shape, strides, dtype=dtype, device="cuda") if strides else \
            torch.zeros(shape, dtype=dtype, device="cuda")
    state = [_i32(a) for a in ([[8, 5], [-1, -1]], [20, 0], [0] * 9, [0, 1, 2, 3, 4, 6, 7, -1, -1], [7])]
    before = [t.clone() for t in state]
    table, lens, shares, free, count = state
    for pools, what in list(_bad(make)) + [([torch.zeros(9, 4)], "on the host")]:
        with pytest.raises(ValueError, match="pools"):
            pa.fork_sequences(_i32([0]), _i32([1]), table, lens, shares, free, count, pools, 16)
        with pytest.raises(ValueError, match="pools"):
            pa.compact_pages(table, lens, shares, free, count, pools, 16)
        assert all(torch.equal(a, b) for a, b in zip(state, before)), what
    assert pa.paged_attn_last_error_word() == 0


@pytest.mark.gpu
def test_many_pools():
    """Four arrays a layer of a hundred layers: every one's pages are copied and moved."""
    import torch
    pa.load_library(build_if_missing=True)
    pools = [torch.randint(-2**31, 2**31 - 1, (9, 1 + i % 7), dtype=torch.int32, device="cuda") for i in range(400)]
    want = [p.clone() for p in pools]
    table, lens, shares, free, count = (_i32(a) for a in ([[8, 5], [-1, -1]], [20, 0], [0] * 9,
                                                          [0, 1, 2, 3, 4, 6, 7, -1, -1], [7]))
    copies = pa.fork_sequences(_i32([0]), _i32([1]), table, lens, shares, free, count, pools, 16)
    assert copies.tolist() == [[5, 7]] and table.tolist() == [[8, 5], [8, 7]]
    for w in want:
        w[7] = w[5]
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    page_map, n = pa.compact_pages(table, lens, shares, free, count, pools, 16)
    assert int(n) == 3 and table.tolist() == [[2, 0], [2, 1]] and int(count) == 6
    for a, b in ((5, 0), (7, 1), (8, 2)):
        for w in want:
            w[b] = w[a]
    assert all(torch.equal(p, w) for p, w in zip(pools, want))
    # without pools the tables change all the same: the caller moves the contents
    assert pa.fork_sequences(_i32([0]), _i32([0]), table, lens, shares, free, count, [], 16).tolist() == [[-1, -1]]
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_REFUSED
