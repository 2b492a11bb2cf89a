"""Refusals of the 4-bit cache's and the page calls: the C ABI's argument checks (nothing is launched) and the
binding's checks of tensors; what the plain implementation of the format holds (CPU only)."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_201_gb300 as pa
from paged_kv_cache_201_gb300 import build
from tests import _kv4_ref as R
from tests.test_serving_step_abi import FakeCuda

OK, EINVAL, EDTYPE, EUNSUP = 0, -1, -2, -3
FAKE = 0x10000  # never dereferenced: every call below fails validation (or has no work) first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pa.load_library()


def _dims(**kw):
    base = dict(batch=2, q_len=3, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=64,
                bt_stride=8, dtype=pa.PA_BF16)
    base.update(kw)
    return pa.PaDims(**base)


def _ref(d):
    return None if d is None else ctypes.byref(_dims(**d))


# ----------------------------------------------------------------------------- the C ABI
@pytest.mark.parametrize("dims,kw,code", [
    (None, {}, EINVAL), (dict(dtype=7), {}, EDTYPE), (dict(head_dim=96), {}, EUNSUP), (dict(page_size=8), {}, EUNSUP),
    (dict(num_pages=1 << 27), {}, EUNSUP), (dict(num_pages=0), {}, EINVAL), (dict(num_kv_heads=3), {}, EINVAL),
    (dict(num_kv_heads=32768, num_q_heads=32768), {}, EUNSUP), ({}, dict(ks=255), EINVAL), ({}, dict(vs=2 * 128 + 4), EINVAL), ({}, dict(ks=1 << 40), EINVAL),
    ({}, dict(k=None), EINVAL), ({}, dict(v=None), EINVAL), ({}, dict(k=FAKE + 8), EINVAL), ({}, dict(kv=None), EINVAL),
    ({}, dict(kv=FAKE + 4), EINVAL), ({}, dict(slots=FAKE + 2), EINVAL), ({}, dict(slots=None), EINVAL),
    (dict(q_len=0), {}, OK), (dict(q_len=0), dict(k=None, v=None, slots=None), OK), (dict(q_len=0, dtype=pa.PA_F32), {}, OK),
])
def test_append_and_gather_refusals(lib, dims, kw, code):
    a = dict(k=FAKE, v=FAKE, slots=FAKE, ks=0, vs=0, kv=FAKE)
    a.update(kw)
    assert lib.paged_attn_append_kv4(a["k"], a["v"], a["slots"], a["ks"], a["vs"], a["kv"], _ref(dims), None) == code
    if "ks" not in kw and "vs" not in kw:
        assert lib.paged_attn_gather_kv4(a["kv"], a["slots"], a["k"], a["v"], _ref(dims), None) == code


@pytest.mark.parametrize("dims,kw,code", [
    (None, {}, EINVAL), (dict(dtype=pa.PA_F32), {}, EDTYPE), (dict(dtype=pa.PA_INT8), {}, EDTYPE),
    (dict(head_dim=32), {}, EUNSUP), (dict(page_size=48), {}, EUNSUP), (dict(num_q_heads=7), {}, EINVAL),
    (dict(num_kv_heads=2**20, num_q_heads=2**20, page_size=64, head_dim=256), {}, EUNSUP),
    ({}, dict(scale=math.nan), EINVAL), ({}, dict(scale=math.inf), EINVAL), ({}, dict(q=None), EINVAL),
    ({}, dict(kv=None), EINVAL), ({}, dict(table=None), EINVAL), ({}, dict(lens=None), EINVAL), ({}, dict(out=None), EINVAL),
    ({}, dict(q=FAKE + 8), EINVAL), ({}, dict(kv=FAKE + 8), EINVAL), ({}, dict(out=FAKE + 8), EINVAL),
    ({}, dict(lse=FAKE + 2), EINVAL), ({}, dict(q_start=FAKE + 2), EINVAL), ({}, dict(q_offset=FAKE + 1), EINVAL),
    ({}, dict(ws=FAKE + 8), EINVAL), ({}, dict(ws_bytes=-1), EINVAL), (dict(q_stride=8 * 128 - 8), {}, EINVAL),
    (dict(q_stride=8 * 128 + 4), {}, EINVAL), (dict(batch=0), {}, OK), (dict(q_len=0), dict(q_start=FAKE), OK),
    (dict(batch=-1), {}, EINVAL),
])
def test_fwd_refusals(lib, dims, kw, code):
    a = dict(q=FAKE, kv=FAKE, table=FAKE, lens=FAKE, q_start=None, q_offset=None, scale=0.1, out=FAKE, lse=FAKE, ws=None,
             ws_bytes=0)
    a.update(kw)
    assert lib.paged_attn_fwd_kv4(a["q"], a["kv"], a["table"], a["lens"], a["q_start"], 1, a["q_offset"], a["scale"],
                                  a["out"], a["lse"], _ref(dims), a["ws"], a["ws_bytes"], None) == code


def test_workspace_bytes(lib):
    """Few rows over long tables make use of a workspace, many rows do not; refusals."""
    f = lambda packed=1, sms=152, **kw: lib.paged_attn_kv4_workspace_bytes(_ref(kw), packed, sms)  # noqa: E731
    row = 8 * 130 * 4
    assert f(batch=1, q_len=1, bt_stride=8192) % row == 0 and f(batch=1, q_len=1, bt_stride=8192) >= 40 * row
    assert f(packed=0, batch=1, q_len=1, bt_stride=8192) == f(batch=1, q_len=1, bt_stride=8192)
    assert f(batch=256, q_len=256, bt_stride=8192) == 0 and f(batch=1, q_len=1, bt_stride=8) == 0
    assert f(batch=1, q_len=300, bt_stride=2000) >= 2 * 300 * row  # a run: tcgen05
    assert f(batch=0, q_len=0) == 0 and f(q_len=0) == 0
    assert f(sms=0) == EINVAL and f(dtype=pa.PA_F32) == EDTYPE and f(head_dim=96) == EUNSUP
    assert lib.paged_attn_kv4_workspace_bytes(None, 1, 152) == EINVAL


COMMON = [(dict(batch=-1), EINVAL), (dict(cap=-1), EINVAL), (dict(width=-1), EINVAL), (dict(num_pages=0), EINVAL),
          (dict(ps=8), EUNSUP), (dict(ps=48), EUNSUP), (dict(num_pages=1 << 27), EUNSUP), (dict(width=1 << 27), EUNSUP),
          (dict(batch=16385), EUNSUP), (dict(lens=None), EINVAL), (dict(table=None), EINVAL), (dict(free=None), EINVAL),
          (dict(count=None), EINVAL), (dict(shares=None), EINVAL), (dict(lens=FAKE + 2), EINVAL),
          (dict(table=FAKE + 1), EINVAL), (dict(shares=FAKE + 2), EINVAL), (dict(free=FAKE + 2), EINVAL)]
BASE = dict(rows=FAKE, children=FAKE, prefix=None, n=3, table=FAKE, lens=FAKE, out=FAKE, shares=FAKE, free=FAKE, cap=9,
            count=FAKE, left=FAKE, copies=FAKE, moves=FAKE, n_moves=FAKE, map=FAKE, batch=4, ps=16, num_pages=64, width=8)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(n=-1), EINVAL), (dict(n=16385), EUNSUP), (dict(n=16384, width=1 << 16), EUNSUP), (dict(rows=None), EINVAL),
    (dict(children=None), EINVAL), (dict(copies=None), EINVAL), (dict(out=None), EINVAL), (dict(left=None), EINVAL),
    (dict(prefix=FAKE + 2), EINVAL), (dict(copies=FAKE + 2), EINVAL),
])
def test_fork_refusals(lib, kw, code):
    a = {**BASE, **kw}
    assert lib.paged_attn_fork(a["rows"], a["children"], a["prefix"], a["n"], a["table"], a["lens"], a["out"], a["shares"],
                               a["free"], a["cap"], a["count"], a["left"], a["copies"], a["batch"], a["ps"],
                               a["num_pages"], a["width"], None) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(n=-1), EINVAL), (dict(n=16385), EUNSUP), (dict(rows=None), EINVAL), (dict(out=None), EINVAL),
    (dict(left=None), EINVAL), (dict(rows=FAKE + 2), EINVAL), (dict(left=FAKE + 2), EINVAL),
])
def test_free_refusals(lib, kw, code):
    a = {**BASE, **kw}
    assert lib.paged_attn_free(a["rows"], a["n"], a["table"], a["lens"], a["out"], a["shares"], a["free"], a["cap"],
                               a["count"], a["left"], a["batch"], a["ps"], a["num_pages"], a["width"], None) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(moves=None), EINVAL), (dict(n_moves=None), EINVAL), (dict(map=None), EINVAL), (dict(moves=FAKE + 2), EINVAL),
    (dict(batch=16384, width=1 << 16), EUNSUP),
])
def test_compact_refusals(lib, kw, code):
    a = {**BASE, **kw}
    assert lib.paged_attn_compact(a["table"], a["lens"], a["shares"], a["free"], a["cap"], a["count"], a["moves"],
                                  a["n_moves"], a["map"], a["batch"], a["ps"], a["num_pages"], a["width"], None) == code


@pytest.mark.parametrize("pools,sizes,kw,code", [
    ([FAKE], [64], dict(num_pages=0), EINVAL), ([FAKE], [64], dict(max_pairs=-1), EINVAL), ([FAKE], [64], dict(n=-1), EINVAL),
    ([FAKE], [6], {}, EINVAL), ([FAKE], [0], {}, EINVAL), ([FAKE + 2], [64], {}, EINVAL), ([None], [64], {}, EINVAL),
    ([FAKE], [1 << 31], {}, EUNSUP), ([FAKE] * 193, [64] * 193, {}, EUNSUP), ([FAKE], [64], dict(pairs=None), EINVAL),
    ([FAKE], [64], dict(pairs=FAKE + 2), EINVAL), ([FAKE], [64], dict(n_pairs=FAKE + 1), EINVAL),
    ([FAKE], [64], dict(num_pages=1 << 31), EUNSUP), ([], [], {}, OK), ([FAKE], [64], dict(max_pairs=0, pairs=None), OK),
])
def test_copy_refusals(lib, pools, sizes, kw, code):
    a = dict(n=len(pools), pairs=FAKE, max_pairs=4, n_pairs=None, num_pages=9)
    a.update(kw)
    p, s = (ctypes.c_void_p * max(1, len(pools)))(*pools), (ctypes.c_int64 * max(1, len(sizes)))(*sizes)
    assert lib.paged_attn_copy_pages(p, s, a["n"], a["pairs"], a["max_pairs"], a["n_pairs"], a["num_pages"], None) == code
    assert lib.paged_attn_copy_pages(None, s, 1, a["pairs"], 1, None, 9, None) == EINVAL


# ----------------------------------------------------------------------------- the binding's checks
@pytest.fixture
def fake_device(monkeypatch):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(pa, "_stream", lambda s: None)
    monkeypatch.setattr(pa, "_sm_count", lambda dev: 152)


def _refused(fn, base, cases):
    for kw, exc in cases:
        with pytest.raises(exc):
            fn(**{**base, **kw})


def test_binding_rows(lib, fake_device):
    import torch
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    cases = [(dict(slots=FakeCuda(4)), ValueError), (dict(slots=FakeCuda(5, dtype=torch.int64)), TypeError),
             (dict(slots=FakeCuda(5, 1)), ValueError), (dict(kv=FakeCuda(9, 2, 16 * 144, dtype=torch.int8)), TypeError),
             (dict(kv=FakeCuda(9, 3, 16 * 144, dtype=u8)), ValueError), (dict(kv=FakeCuda(9, 2, 16 * 145, dtype=u8)), ValueError),
             (dict(kv=FakeCuda(9, 2, 8 * 144, dtype=u8)), ValueError), (dict(kv=FakeCuda(9, 2, 16, 144, dtype=u8)), ValueError),
             (dict(slots=FakeCuda(5, device=1)), ValueError), (dict(slots=torch.zeros(5, dtype=torch.int32)), ValueError)]
    base = dict(k_new=FakeCuda(5, 2, 128, dtype=bf), v_new=FakeCuda(5, 2, 128, dtype=bf), slots=FakeCuda(5),
                kv=FakeCuda(9, 2, 16 * 144, dtype=u8))
    _refused(pa.paged_attn_append_kv4, base, cases + [
        (dict(k_new=FakeCuda(4, 2, 128, dtype=bf)), ValueError), (dict(v_new=FakeCuda(5, 2, 128, dtype=f32)), TypeError),
        (dict(k_new=FakeCuda(5, 2, 128, dtype=torch.float64), v_new=FakeCuda(5, 2, 128, dtype=torch.float64)), TypeError),
        (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, strides=(0, 128, 1))), ValueError),
        (dict(v_new=FakeCuda(5, 2, 128, dtype=bf, strides=(256, 1, 2))), ValueError),
        (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, strides=(260, 128, 1))), pa.PagedAttnError),
        (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, device=1)), ValueError),
        (dict(k_new=torch.zeros(5, 2, 128, dtype=bf)), ValueError)])
    base = dict(kv=base["kv"], slots=base["slots"], k_out=base["k_new"], v_out=base["v_new"])
    _refused(pa.paged_attn_gather_kv4, base, cases + [
        (dict(k_out=FakeCuda(5, 2, 128, dtype=bf, strides=(512, 128, 1))), ValueError),
        (dict(v_out=FakeCuda(5, 2, 64, dtype=bf)), ValueError), (dict(v_out=FakeCuda(5, 2, 128, dtype=f32)), TypeError)])


def test_binding_fwd(lib, fake_device):
    import torch
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    base = dict(q=FakeCuda(7, 8, 128, dtype=bf), kv=FakeCuda(9, 2, 16 * 144, dtype=u8), block_table=FakeCuda(3, 6),
                seq_lens=FakeCuda(3), causal=True, q_offset=None, scale=0.1, out=FakeCuda(7, 8, 128, dtype=bf),
                lse=FakeCuda(7, 8, dtype=f32), q_start=FakeCuda(4))
    _refused(pa.paged_attn_fwd_kv4, base, [
        (dict(q=FakeCuda(7, 8, 64, dtype=bf)), ValueError), (dict(q=FakeCuda(1, 7, 8, 128, dtype=bf)), ValueError),
        (dict(q_start=None), ValueError), (dict(q_start=FakeCuda(3)), ValueError), (dict(seq_lens=FakeCuda(4)), ValueError),
        (dict(q_offset=FakeCuda(2)), ValueError), (dict(kv=FakeCuda(9, 2, 16 * 144, dtype=bf)), TypeError),
        (dict(kv=FakeCuda(9, 3, 16 * 144, dtype=u8)), pa.PagedAttnError),  # 8 heads over 3
        (dict(out=FakeCuda(7, 8, 128, dtype=f32)), TypeError), (dict(out=FakeCuda(7, 4, 128, dtype=bf)), ValueError),
        (dict(lse=FakeCuda(7, 2, dtype=f32)), ValueError), (dict(scale=math.nan), pa.PagedAttnError),
        (dict(q=FakeCuda(7, 8, 128, dtype=bf, strides=(0, 128, 1))), ValueError),
        (dict(block_table=FakeCuda(3, 6, device=1)), ValueError), (dict(workspace=FakeCuda(64, dtype=f32)), TypeError),
        (dict(q=FakeCuda(7, 8, 128, dtype=f32), out=FakeCuda(7, 8, 128, dtype=f32)), pa.PagedAttnError)])


def test_binding_pages(lib, fake_device):
    import torch
    state = dict(block_table=FakeCuda(4, 6), seq_lens=FakeCuda(4), page_shares=FakeCuda(9), free_pages=FakeCuda(9),
                 free_count=FakeCuda(1), page_size=16)
    cases = [(dict(block_table=FakeCuda(4, 6, device=1)), ValueError), (dict(seq_lens=FakeCuda(5)), ValueError),
             (dict(page_shares=FakeCuda(9, dtype=torch.int64)), TypeError), (dict(page_shares=FakeCuda(9, 1)), ValueError),
             (dict(free_pages=FakeCuda(9, strides=(2,))), ValueError), (dict(free_count=FakeCuda(2)), ValueError),
             (dict(page_size=8), pa.PagedAttnError), (dict(block_table=torch.zeros(4, 6, dtype=torch.int32)), ValueError)]
    outs = dict(lens_out=FakeCuda(4), free_left=FakeCuda(1))
    more = [(dict(lens_out=FakeCuda(3)), ValueError), (dict(free_left=FakeCuda(1, dtype=torch.float32)), TypeError)]
    _refused(pa.paged_attn_fork, dict(parents=FakeCuda(3), children=FakeCuda(3), copies=FakeCuda(3, 2), **state, **outs),
             cases + more + [(dict(children=FakeCuda(2)), ValueError), (dict(copies=FakeCuda(3)), ValueError),
                             (dict(prefix_lens=FakeCuda(4)), ValueError), (dict(parents=FakeCuda(3, 1)), ValueError)])
    _refused(pa.paged_attn_free, dict(rows=FakeCuda(3), **state, **outs),
             cases + more + [(dict(rows=FakeCuda(3, dtype=torch.int64)), TypeError), (dict(rows=FakeCuda(3, 1)), ValueError)])
    _refused(pa.paged_attn_compact, dict(moves=FakeCuda(4, 2), n_moves=FakeCuda(1), page_map=FakeCuda(9), **state),
             cases + [(dict(moves=FakeCuda(3, 2)), ValueError), (dict(page_map=FakeCuda(8)), ValueError),
                      (dict(n_moves=FakeCuda(2)), ValueError)])
    pools = [FakeCuda(9, 4, dtype=torch.float32), FakeCuda(9, 2, 8, dtype=torch.uint8)]
    _refused(pa.paged_attn_copy_pages, dict(pools=pools, pairs=FakeCuda(5, 2)), [
        (dict(pools=[]), ValueError), (dict(pools=[pools[0], FakeCuda(8, 4)]), ValueError), (dict(pairs=FakeCuda(5, 3)), ValueError),
        (dict(pairs=FakeCuda(5)), ValueError), (dict(n_pairs=FakeCuda(2)), ValueError),
        (dict(pools=[FakeCuda(9, 4, strides=(8, 1))]), ValueError), (dict(pools=[FakeCuda(9, 3, dtype=torch.uint8)]), pa.PagedAttnError),
        (dict(pools=[FakeCuda(9, 4, device=1)]), ValueError), (dict(pools=[FakeCuda(9)]), ValueError)])


# ----------------------------------------------------------------------------- the format
def test_scales_are_f16_numbers():
    bits = (np.arange(0xDF, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(bits, R.SCALES)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_are_nearest(D):
    """No other code of its scale is nearer to an element, no other scale to a seventh of the largest."""
    rng = np.random.default_rng(D)
    x = rng.standard_normal((40, D)) * np.exp(rng.uniform(-13, 9, (40, 1)))
    u, c = R.quantise(x)
    g, s = x.reshape(40, -1, 16), R.SCALES[c.astype(int)]
    best = np.abs(g[..., None] - s[..., None, None] * np.arange(-7, 8)).min(-1)
    held = (u.reshape(g.shape).astype(float) - 8) * s[..., None]
    np.testing.assert_allclose(np.abs(g - held), best, rtol=1e-12, atol=1e-12 * np.abs(g).max())
    t = np.abs(g).max(-1, keepdims=True) / 7
    assert (np.abs(s - t[..., 0]) <= np.abs(R.SCALES - t).min(-1) * (1 + 1e-12)).all()


def test_pool_layout():
    """A row's bytes stand where the header says: codes of K, of V, scales of K, of V, elements in nibbles."""
    ps, D = 16, 64
    pool = np.zeros((3, 2, 9 * ps * D // 8), np.uint8)
    k, v = np.zeros((1, 2, D)), np.zeros((1, 2, D))
    k[0, 1, 17], v[0, 1, 18] = 7.0, -14.0  # scales 1 and 2: bytes 120 and 128
    R.write(pool, [2 * ps + 5], k, v, ps)
    block = pool[2, 1]
    assert block[5 * 32 + 8] == 0x88 | 0x70 and block[ps * 32 + 5 * 32 + 9] == 0x81
    assert block[ps * D + 5 * 4 + 1] == 120 and block[ps * D + ps * 4 + 5 * 4 + 1] == 128
    kk, vv = R.values(pool, ps, D)
    assert kk[2, 1, 5, 17] == 7.0 and vv[2, 1, 5, 18] == -14.0 and np.abs(kk).sum() == 7.0 and np.abs(vv).sum() == 14.0


def test_short_way_refuses_what_is_no_tensor(lib):
    """What is not as it should be goes the long way, which says what: the short one says nothing."""
    import torch
    short = pa._short()
    arity = dict(append_kv4=5, gather_kv4=5, fwd_kv4=12, fork=13, free=10, compact=10, copy_pages=4)
    host = torch.zeros((3, 2, 64))
    for name, n in arity.items():
        fn = getattr(short, name)
        assert fn(*[None] * n) is None and fn(*[host] * n) is None and fn(*[FakeCuda(3, 2)] * n) is None
        with pytest.raises(TypeError):
            fn(*[None] * (n + 1))
    assert short.copy_pages([host] * 3, torch.zeros((2, 2), dtype=torch.int32), None, None) is None
