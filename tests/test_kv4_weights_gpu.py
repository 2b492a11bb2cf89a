"""Attention over the 4-bit cache where the weighted values cancel: keys come in pairs whose V rows are x and -x
and whose scores nearly agree, so an output is much smaller than the mean of |v| that its weights are off by.

The bar is that of tests/test_kv4_gpu.py for weights of two f16 numbers, whatever the output's type: half a rounding step of
the output, what float32 sums may lose in the scores, and 2^-22 of sum w |v| / sum w for the weights.
One f16 number, off by up to 2^-12 of a weight just below a power of two, misses it."""
import numpy as np
import pytest

from tests import _kv4_ref as R

pytestmark = pytest.mark.gpu

STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_201_gb300 as pa
    pa.load_library(build_if_missing=True)
    pa.paged_attn_last_error_word()
    return pa


def _check(pa, lens, new, Hkv, G, D, ps, dtype, width=None, workspace=True, packed=True):
    import torch
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    rng = np.random.default_rng(sum(lens) + G * D)
    lens, new = np.asarray(lens), np.asarray(new)
    need = -(-lens // ps)
    P = int(need.sum())
    table = np.zeros((len(lens), width or int(need.max())), np.int32)
    table[np.arange(table.shape[1])[None] < need[:, None]] = rng.permutation(P)
    slots = np.concatenate([table[b, np.arange(n) // ps] * ps + np.arange(n) % ps for b, n in enumerate(lens)])
    k, v = rng.standard_normal((2, len(slots), Hkv, D))
    at = np.concatenate([[0], np.cumsum(lens)])
    for a, n in zip(at, lens):  # every second V row is its predecessor's negative
        v[a + 1:a + n - n % 2:2] = -v[a:a + n - n % 2:2]
    pool = np.zeros((P, Hkv, 9 * ps * D // 8), np.uint8)
    R.write(pool, slots, k, v, ps)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(0.003 * rng.standard_normal((starts[-1], Hkv * G, D))).to(dt).cuda()
    gpu = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    shape = q.shape if packed else (len(lens), -1, *q.shape[1:])
    pa.paged_attn_fwd_kv4(q.view(shape), torch.from_numpy(pool).cuda(), gpu(table), gpu(lens), False, None, D ** -0.5,
                          out.view(shape), lse.view(shape[:-1]), q_start=gpu(starts) if packed else None,
                          workspace=None if workspace else torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert pa.paged_attn_last_error_word() == 0
    want, want_lse, off, room, mass = R.attention(q.double().cpu().numpy(), pool, ps, table, lens, starts, False, None, D ** -0.5)
    bar = STEP[dtype] * np.abs(want) + room + 2.0 ** -22 * mass + 2.0 ** -24
    worst = np.abs(out.double().cpu().numpy() - want) / bar
    assert worst.max() <= 1, f"output off by {worst.max():.3g} of its bar"
    worst = np.abs(lse.double().cpu().numpy() - want_lse) / (off + 2.0 ** -22 * np.abs(want_lse))
    assert worst.max() <= 1, f"lse off by {worst.max():.3g} of its bar"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 12, 40])
def test_single_tokens(pa, G, D, dtype):
    _check(pa, [2, 4, 16, 40, 200], [1] * 5, 2, G, D, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Sq,G,D", [(1, 4, 128), (2, 2, 64), (4, 1, 128), (3, 1, 256), (1, 5, 128), (5, 1, 64), (2, 3, 256)])
def test_uniform(pa, Sq, G, D, dtype):
    """Up to four rows a unit and more."""
    _check(pa, [6, 40, 130], [Sq] * 3, 2, G, D, 32, dtype, packed=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_keys_shared(pa, dtype):
    """By a cluster, and by a grid's CTAs."""
    for workspace in (False, True):
        _check(pa, [600], [1], 2, 4, 128, 32, dtype, width=512, workspace=workspace)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,new,G", [([300, 150, 64], [100, 70, 1], 8), ([200], [65], 3), ([1500], [130], 4)])
def test_runs(pa, lens, new, G, D, dtype):
    """On tcgen05, with single tokens beside them, and with few tiles over many keys."""
    _check(pa, lens, new, 1, G, D, 16, dtype, width=None if len(lens) > 1 else 200)
