"""Rows of long prompts into a 4-bit pool and back, where a thread takes four of them: skipped and bad slots among a
thread's rows, rows left over at the end, inputs further apart than their heads.  Bit for bit."""
import numpy as np
import pytest

from tests import _kv4_ref as R
from tests.test_kv4_gpu import _dt, _np, _rows, _t, pa  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,Hkv,T,ps", [(64, 8, 8203, 16), (128, 8, 4099, 64), (256, 8, 2051, 32), (128, 3, 10931, 16),
                                        (64, 5, 13111, 64), (256, 1, 16387, 16)])
def test_rows_of_prompts(pa, D, Hkv, T, ps, dtype):
    import torch
    assert T * Hkv * D // 8 >= 1 << 19  # from here on a thread takes four rows
    rng = np.random.default_rng(T + D)
    P = -(-T // ps) + 3
    slots = rng.permutation(P * ps)[:T].astype(np.int32)
    slots[rng.uniform(size=T) < 0.1] = -1
    slots[rng.integers(0, T, 40)] = -1
    bad = rng.permutation(T)[:30]
    slots[bad] = rng.choice([P * ps, P * ps + 7, -2, 2**31 - 1, -2**31], 30)
    slots[-1], slots[0] = P * ps, -1
    wide = _rows(rng, (T, 2 * Hkv + 1, D), dtype)
    k, v = wide[:, :Hkv], wide[:, Hkv:2 * Hkv]
    kv = torch.randint(0, 256, (P, Hkv, 9 * ps * D // 8), dtype=torch.uint8, device="cuda")
    want = kv.cpu().numpy().copy()
    x, y = _np(k), _np(v)
    for n in (T, T - 37):  # and with another remainder
        pa.paged_attn_append_kv4(k[:n], v[:n], _t(slots[:n]), kv)
        assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE
        if n == T:
            R.write(want, slots, x, y, ps)
        np.testing.assert_array_equal(kv.cpu().numpy(), want)
    got_k, got_v = (torch.full((T, Hkv, D), 7.0, dtype=_dt(dtype), device="cuda") for _ in "kv")
    pa.paged_attn_gather_kv4(kv, _t(slots), got_k, got_v)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE
    good = (slots >= 0) & (slots < P * ps)
    for got, held in zip((got_k, got_v), R.values(want, ps, D)):
        held = held.transpose(0, 2, 1, 3).reshape(P * ps, Hkv, D)[np.where(good, slots, 0)]
        np.testing.assert_array_equal(_np(got), np.where(good[:, None, None], held, 0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompts_not_finite(pa, dtype):
    """NaN and infinities in any of a thread's four rows."""
    import torch
    rng = np.random.default_rng(9)
    T, Hkv, D = 4099, 8, 128
    k, v = _rows(rng, (T, Hkv, D), dtype), _rows(rng, (T, Hkv, D), dtype)
    for i, bad in enumerate((np.nan, np.inf, -np.inf)):
        k[i::1001, i, 30 + i], v[5 + i::37, 7 - i, 3 * i] = bad, bad
    kv = pa.kv4_pool(-(-T // 16), 16, Hkv, D)
    want = kv.cpu().numpy()
    slots = np.arange(T, dtype=np.int32)
    pa.paged_attn_append_kv4(k, v, _t(slots), kv)
    assert pa.paged_attn_last_error_status() == (pa.PA_OK, pa.ERRBIT_NONFINITE)
    R.write(want, slots, _np(k), _np(v), 16)
    np.testing.assert_array_equal(kv.cpu().numpy(), want)
