"""Refusals of the serving-step calls: the C ABI's argument checks (nothing is launched) and the
binding's checks of tensors (CPU only)."""
import ctypes
import math

import pytest

import paged_kv_cache_201_gb300 as pa
from paged_kv_cache_201_gb300 import build

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
    return None if d is None else ctypes.byref(d)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), EINVAL), (dict(total=-1), EINVAL), (dict(cap=-1), EINVAL), (dict(width=-1), EINVAL),
    (dict(num_pages=0), EINVAL), (dict(ps=8), EUNSUP), (dict(ps=48), EUNSUP), (dict(num_pages=1 << 27), EUNSUP),
    (dict(width=1 << 27), EUNSUP), (dict(batch=16385), EUNSUP), (dict(batch=0), OK), (dict(cached=None), EINVAL),
    (dict(free=None), EINVAL), (dict(table=None), EINVAL), (dict(slots=None), EINVAL), (dict(slots=FAKE + 2), EINVAL),
    (dict(left=None), EINVAL), (dict(q_start=FAKE + 1), EINVAL),
])
def test_step_tables_refusals(lib, kw, code):
    a = dict(cached=FAKE, new=FAKE, free=FAKE, cap=5, count=FAKE, table=FAKE, lens=FAKE, q_offset=FAKE, q_start=FAKE,
             slots=FAKE, left=FAKE, batch=4, total=9, ps=16, num_pages=64, width=8)
    a.update(kw)
    assert lib.paged_attn_step_tables(a["cached"], a["new"], a["free"], a["cap"], a["count"], a["table"], a["lens"],
                                      a["q_offset"], a["q_start"], a["slots"], a["left"], a["batch"], a["total"],
                                      a["ps"], a["num_pages"], a["width"], None) == code


@pytest.mark.parametrize("dims,kw,code", [
    (None, {}, EINVAL), (dict(dtype=7), {}, EDTYPE), (dict(head_dim=96), {}, EUNSUP), (dict(page_size=8), {}, EUNSUP),
    ({}, dict(ks=255), EINVAL), ({}, dict(vs=2 * 128 + 4), EINVAL), ({}, dict(ks=1 << 40), EINVAL),
    ({}, dict(k=None), EINVAL), ({}, dict(k=FAKE + 8), EINVAL), ({}, dict(vc=FAKE + 2), EINVAL),
    ({}, dict(env=FAKE), EINVAL), ({}, dict(scale=FAKE), EINVAL), ({}, dict(env=FAKE + 8, scale=FAKE), EINVAL),
    ({}, dict(env=FAKE, scale=FAKE + 2), EINVAL), ({}, dict(slots=FAKE + 2), EINVAL), (dict(q_len=0), {}, OK),
    (dict(q_len=0), dict(ks=3 * 2 * 128), OK), (dict(num_pages=1 << 27), {}, EUNSUP),
])
def test_append_refusals(lib, dims, kw, code):
    a = dict(k=FAKE, v=FAKE, slots=FAKE, ks=0, vs=0, kc=FAKE, vc=FAKE, env=None, scale=None)
    a.update(kw)
    d = None if dims is None else _dims(**dims)
    assert lib.paged_attn_append(a["k"], a["v"], a["slots"], a["ks"], a["vs"], a["kc"], a["vc"], a["env"], a["scale"],
                                 _ref(d), None) == code


@pytest.mark.parametrize("dims,kw,code", [
    (None, {}, EINVAL), (dict(dtype=3), {}, EDTYPE), (dict(head_dim=32), {}, EUNSUP), ({}, dict(K=0), EINVAL),
    ({}, dict(sink=-1), EINVAL), ({}, dict(local=-1), EINVAL), ({}, dict(sink=3, local=2), EINVAL),
    ({}, dict(sink=2**31 - 1, local=2**31 - 1), EINVAL), (dict(bt_stride=49153), {}, EUNSUP),
    (dict(num_q_heads=7), {}, EINVAL), ({}, dict(env=None), EINVAL), ({}, dict(env=FAKE + 8), EINVAL),
    ({}, dict(scale=None), EINVAL), ({}, dict(q=FAKE + 8), EINVAL), ({}, dict(sel=None), EINVAL),
    ({}, dict(sel=FAKE + 2), EINVAL), ({}, dict(q_start=FAKE + 2), EINVAL), (dict(batch=0), {}, OK),
    ({}, dict(K=(1 << 24) + 1), EUNSUP), (dict(q_len=0), {}, OK), (dict(q_stride=8 * 128 - 8), {}, EINVAL),
])
def test_select_refusals(lib, dims, kw, code):
    a = dict(q=FAKE, env=FAKE, scale=FAKE, table=FAKE, lens=FAKE, q_start=None, sink=1, local=1, K=4, sel=FAKE)
    a.update(kw)
    d = None if dims is None else _dims(**dims)
    assert lib.paged_attn_select_pages(a["q"], a["env"], a["scale"], a["table"], a["lens"], a["q_start"], 1, None,
                                       a["sink"], a["local"], a["K"], a["sel"], _ref(d), None) == code


@pytest.mark.parametrize("dims,kw,code", [
    (None, {}, EINVAL), (dict(dtype=pa.PA_INT8), {}, EDTYPE), (dict(head_dim=96), {}, EUNSUP), ({}, dict(K=0), EINVAL),
    ({}, dict(factor=math.nan), EINVAL), ({}, dict(factor=math.inf), EINVAL), ({}, dict(k=None), EINVAL),
    ({}, dict(out=FAKE + 8), EINVAL), ({}, dict(lse=FAKE + 2), EINVAL), ({}, dict(sel=FAKE + 2), EINVAL),
    ({}, dict(table=None), EINVAL), (dict(batch=0), {}, OK), (dict(q_len=0), dict(lse=None), OK),
    ({}, dict(K=(1 << 24) + 1), EUNSUP),
])
def test_sparse_refusals(lib, dims, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, q_start=None, sel=FAKE, K=4, factor=0.1, out=FAKE,
             lse=FAKE)
    a.update(kw)
    d = None if dims is None else _dims(**dims)
    assert lib.paged_attn_fwd_sparse(a["q"], a["k"], a["v"], a["table"], a["lens"], a["q_start"], 1, None, a["sel"],
                                     a["K"], a["factor"], a["out"], a["lse"], _ref(d), None) == code


def test_sparse_kernel_choice(lib):
    """Runs of many tokens share page loads; single tokens, short runs, f32, head_dim 256, scale <= 0, wide
    tables and over 128 query heads to a kv head do not."""
    f = lambda scale=0.1, K=64, sms=152, packed=1, **kw: lib.paged_attn_sparse_shares_pages(  # noqa: E731
        _ref(_dims(**{**dict(batch=2, q_len=1024, num_q_heads=32, num_kv_heads=8, bt_stride=512), **kw})), packed, K,
        scale, sms)
    assert f() == 1 and f(dtype=pa.PA_F16) == 1 and f(packed=0) == 1
    assert f(q_len=64) == 0 and f(batch=600) == 0 and f(packed=0, q_len=15, batch=300) == 0
    assert f(dtype=pa.PA_F32) == 0 and f(head_dim=256) == 0 and f(scale=0.0) == 0 and f(scale=-1.0) == 0
    assert f(bt_stride=4609, q_len=100000) == 0 and f(num_q_heads=129, num_kv_heads=1) == 0
    assert f(K=0) == EINVAL and f(sms=0) == EINVAL and f(head_dim=96) == EUNSUP
    assert lib.paged_attn_sparse_shares_pages(None, 1, 4, 0.1, 152) == EINVAL


# ----------------------------------------------------------------------------- the binding's checks
class FakeCuda:
    """Enough of a CUDA tensor for the binding's checks; its pointer is never read."""

    def __init__(self, *shape, dtype=None, strides=None, device=0):
        import torch
        self.t = torch.empty(shape, dtype=dtype or torch.int32, device="meta")
        if strides:
            self.t = torch.empty_strided(shape, strides, dtype=dtype or torch.int32, device="meta")
        self.shape, self.dtype, self.is_cuda, self.index = self.t.shape, self.t.dtype, True, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return FAKE


@pytest.fixture
def fake_device(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(pa, "_stream", lambda s: None)


def _tables_args(**kw):
    a = dict(cached_lens=FakeCuda(4), new_lens=FakeCuda(4), free_pages=FakeCuda(9), free_count=FakeCuda(1),
             block_table=FakeCuda(4, 8), seq_lens=FakeCuda(4), q_offset=FakeCuda(4), q_start=FakeCuda(5),
             slots=FakeCuda(20), free_left=FakeCuda(1), page_size=16, num_pages=64)
    a.update(kw)
    return a


def test_binding_step_tables(lib, fake_device):
    import torch
    for kw, exc in [(dict(cached_lens=FakeCuda(3)), ValueError), (dict(q_start=FakeCuda(4)), ValueError),
                    (dict(free_left=FakeCuda(2)), ValueError), (dict(slots=FakeCuda(20, dtype=torch.int64)), TypeError),
                    (dict(new_lens=FakeCuda(4, strides=(2,))), ValueError), (dict(slots=torch.zeros(3)), ValueError),
                    (dict(seq_lens=FakeCuda(4, device=1)), ValueError), (dict(page_size=8), pa.PagedAttnError)]:
        with pytest.raises(exc):
            pa.paged_attn_step_tables(**_tables_args(**kw))


def test_binding_append(lib, fake_device):
    import torch
    bf, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    base = dict(k_new=FakeCuda(5, 2, 128, dtype=bf), v_new=FakeCuda(5, 2, 128, dtype=bf), slots=FakeCuda(5),
                k_cache=FakeCuda(9, 16, 2, 128, dtype=bf), v_cache=FakeCuda(9, 16, 2, 128, dtype=bf),
                k_env=FakeCuda(9, 2, 2, 128, dtype=i8), k_env_scale=FakeCuda(9, 2, dtype=f32))
    for kw, exc in [(dict(k_new=FakeCuda(4, 2, 128, dtype=bf)), ValueError),
                    (dict(k_new=FakeCuda(5, 2, 64, dtype=bf)), ValueError),
                    (dict(v_new=FakeCuda(5, 2, 128, dtype=f32)), TypeError),
                    (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, strides=(0, 128, 1))), ValueError),  # broadcast
                    (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, strides=(128, 128, 1))), ValueError),
                    (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, strides=(256, 1, 2))), ValueError),
                    (dict(k_new=FakeCuda(5, 2, 128, dtype=bf, strides=(260, 128, 1))), pa.PagedAttnError),
                    (dict(k_env=None), ValueError), (dict(k_env=FakeCuda(9, 2, 128, dtype=i8)), ValueError),
                    (dict(k_env=FakeCuda(8, 2, 2, 128, dtype=i8)), ValueError),
                    (dict(k_env_scale=FakeCuda(9, 3, dtype=f32)), ValueError),
                    (dict(slots=FakeCuda(5, device=1)), ValueError),
                    (dict(v_cache=FakeCuda(9, 16, 1, 128, dtype=bf)), ValueError)]:
        with pytest.raises(exc):
            pa.paged_attn_append(**{**base, **kw})


def test_binding_select_and_sparse(lib, fake_device):
    import torch
    bf, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    common = dict(q=FakeCuda(7, 8, 128, dtype=bf), block_table=FakeCuda(3, 6), seq_lens=FakeCuda(3), causal=True,
                  q_offset=None, sel=FakeCuda(7, 2, 4), q_start=FakeCuda(4))
    sel = dict(k_env=FakeCuda(9, 2, 2, 128, dtype=i8), k_env_scale=FakeCuda(9, 2, dtype=f32), sink_pages=1,
               local_pages=1, page_size=16)
    att = dict(k_cache=FakeCuda(9, 16, 2, 128, dtype=bf), v_cache=FakeCuda(9, 16, 2, 128, dtype=bf), scale=0.1,
               out=FakeCuda(7, 8, 128, dtype=bf), lse=FakeCuda(7, 8, dtype=f32))
    bad = [(dict(q=FakeCuda(7, 8, 64, dtype=bf)), ValueError), (dict(q=FakeCuda(1, 7, 8, 128, dtype=bf)), ValueError),
           (dict(q_start=FakeCuda(3)), ValueError), (dict(q_start=None), ValueError),
           (dict(seq_lens=FakeCuda(4)), ValueError), (dict(q_offset=FakeCuda(2)), ValueError),
           (dict(sel=FakeCuda(7, 3, 4)), ValueError), (dict(sel=FakeCuda(6, 2, 4)), ValueError),
           (dict(sel=FakeCuda(7, 2, 4, dtype=torch.int64)), TypeError),
           (dict(q=FakeCuda(7, 8, 128, dtype=bf, strides=(0, 128, 1))), ValueError),
           (dict(q=FakeCuda(7, 8, 128, dtype=bf, strides=(512, 128, 1))), ValueError),
           (dict(block_table=FakeCuda(3, 6, device=1)), ValueError), (dict(sel=FakeCuda(7, 2, 0)), pa.PagedAttnError)]
    for kw, exc in bad + [(dict(sink_pages=4), pa.PagedAttnError), (dict(page_size=12), pa.PagedAttnError),
                          (dict(k_env_scale=FakeCuda(9, 1, dtype=f32)), ValueError)]:
        with pytest.raises(exc):
            pa.paged_attn_select_pages(**{**common, **sel, **kw})
    for kw, exc in bad + [(dict(out=FakeCuda(7, 8, 128, dtype=f32)), TypeError), (dict(scale=math.inf), pa.PagedAttnError),
                          (dict(out=FakeCuda(7, 4, 128, dtype=bf)), ValueError),
                          (dict(lse=FakeCuda(7, 2, dtype=f32)), ValueError),
                          (dict(v_cache=FakeCuda(9, 16, 2, 64, dtype=bf)), ValueError)]:
        with pytest.raises(exc):
            pa.paged_attn_fwd_sparse(**{**common, **att, **kw})
