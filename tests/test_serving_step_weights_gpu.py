"""The weights of the sparse attention in f16: keys far below a row's largest weight count in full.

One sink key has the row's largest score and a value of zero; every other key's score lies x powers of two
(spread 0.3) below it and its value is large, so the output is the sum of the small weights alone.

What a kernel may be off by, for weights w_j = 2^-x_j (the sink's is 1) and l = sum w_j:
  - the rounding of the output to f16: 2^-11 |o|;
  - the weights: a score of at most 32 in log2 units rounded to float32 (2^-20 ln 2), ex2.approx (2^-22) and an
    f16 pair (2^-20): together below 2^-18 |o|;
  - an f16 pair's quantum of 2^-24, half of it for each weight, where a row's largest weight is held as 2^10 at
    least: 2^-35 sum |v_j| / l;
  - float32 sums of n terms, in o and in l: 2 n 2^-24 |o|.
"""
import numpy as np
import pytest

from paged_kv_cache_201_gb300 import workloads as W
from tests import _gpu
from tests import _sparse_ref as R
from tests.test_serving_step_gpu import _check_attend, _lists, _run_attend, _shares, pa  # noqa: F401

pytestmark = pytest.mark.gpu

LN2 = float(np.log(2.0))  # as the scale: scores are then powers of two


def _sink_batch(q_lens, n, D, Hq, Hkv, x, sink, seed):
    b = R.Batch(seed, q_lens, [n] * len(q_lens), Hq, Hkv, D, 16, "f16")
    rng = np.random.default_rng(seed)
    k, v = b.k.view(np.float16), b.v.view(np.float16)
    q = b.q.view(np.float16)
    q[..., 0] = 1.0
    k[:] = 0.0
    k[..., 0] = -rng.normal(x, 0.3, k.shape[:-1])
    v[:] = rng.uniform(3e4, 6e4, v.shape)
    for s in range(len(q_lens)):
        page, row = b.table[s, sink // 16], sink % 16
        k[page, row, :, 0] = 0.0
        v[page, row] = 0.0
    return b


def _check_sink(pa, b, n, sel, **kw):
    out, lse = _run_attend(pa, b, sel, causal=False, scale=LN2, **kw)
    k, v = R.elems_to_f64(b.k, "f16"), R.elems_to_f64(b.v, "f16")
    want, want_lse = R.attend(b.q64(), k, v, b.table, b.rows(causal=False), sel, 16, LN2)
    w_sum = np.exp(want_lse)[..., None]  # the sink's weight is 1
    floor = 2.0 ** -35 * np.abs(v).max() * n / w_sum
    bound = (2.0 ** -11 + 2.0 ** -18 + 2 * n * 2.0 ** -24) * np.abs(want) + floor
    err = np.abs(out - want)
    assert (err <= bound).all(), f"worst: {(err / bound).max():.3g} of the bound, {(err / want).max():.3g} of the output"
    assert np.abs(lse - want_lse).max() < 1e-5


@pytest.mark.parametrize("x", [14, 17, 20, 24, 25])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("sink", [0, 1023])
def test_small_weights_runs_of_tokens(pa, D, Hq, Hkv, x, sink):  # noqa: F811
    """The kernel that reads the union of a run's lists; the sink in the first tile or in the last."""
    n = 1024
    b = _sink_batch([256, 256], n, D, Hq, Hkv, x, sink, x)
    sel = np.broadcast_to(np.arange(n // 16, dtype=np.int32), (b.T, Hkv, n // 16)).copy()
    assert _shares(pa, b, n // 16, scale=LN2)
    _check_sink(pa, b, n, sel)


@pytest.mark.parametrize("x", [14, 17, 20, 24, 25])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 3, 3), (256, 6, 2)])
@pytest.mark.parametrize("q_lens", [[1], [1] * 40])
def test_small_weights_single_tokens(pa, D, Hq, Hkv, x, q_lens):  # noqa: F811
    """The kernel that reads a token's own list, split over a cluster or not."""
    n = 1024
    b = _sink_batch(q_lens, n, D, Hq, Hkv, x, 37, x)
    sel = np.broadcast_to(np.arange(n // 16, dtype=np.int32), (b.T, Hkv, n // 16)).copy()
    assert not _shares(pa, b, n // 16, scale=LN2)
    _check_sink(pa, b, n, sel)


@pytest.mark.parametrize("q_lens", [[1, 1], [200, 200]])
def test_large_scores(pa, q_lens):  # noqa: F811
    """Scores up to 2^13 apart, the largest met late: the weights' scaling follows the maximum."""
    b = R.Batch(5, q_lens, [700, 650], 8, 2, 128, 16, "f16")
    sel = _lists(b, 44)
    for scale in (1.0, 30.0):
        _check_attend(pa, b, sel, scale=scale)
