"""The 4-bit cache on the GPU: rows quantised into a pool and read back (bit for bit), and attention over
the pool against 64-bit arithmetic on the values its bytes stand for.

Attention's bars are derived, not fitted: half a rounding step of the output type (bf16 2^-8, f16 2^-11,
relative) on top of what float32 sums may lose in the scores, which tests/_kv4_ref.py works out row by row from the
inputs, and what the weights lose on their way to V: sum w |v| / sum w times half an f16 step, 2^-11, where they
are one f16 number (bf16 outputs), the square of it where they are two.
"""
import numpy as np
import pytest

from tests import _kv4_ref as R

pytestmark = pytest.mark.gpu

STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
WEIGHT = {"bf16": 2.0 ** -11, "f16": 2.0 ** -22}


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_201_gb300 as pa
    pa.load_library(build_if_missing=True)
    pa.paged_attn_last_error_word()
    return pa


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _t(a, dtype=None):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _rows(rng, shape, dtype):
    """Rows with groups of very different sizes, zeros among them, and values on the borders between codes."""
    import torch
    x = rng.standard_normal(shape) * np.exp(rng.uniform(-12, 6, (*shape[:-1], 1)))
    x[rng.uniform(size=shape) < 0.1] = 0
    g = x.reshape(*shape[:-1], -1, 16)
    g[rng.uniform(size=g.shape[:-1]) < 0.1] = 0
    tie = rng.uniform(size=g.shape[:-1]) < 0.3  # a group of halves of a power of two: a scale of 1 or 9/8 ...
    g[tie] = (rng.integers(-15, 16, g[tie].shape) / 2.0) * 2.0 ** rng.integers(-16, 9, (tie.sum(), 1))
    return torch.from_numpy(x).to(_dt(dtype)).cuda()


# ----------------------------------------------------------------------------- rows
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hkv,ps", [(1, 1, 16), (37, 3, 32), (130, 8, 64), (300, 2, 16)])
def test_rows(pa, T, Hkv, D, ps, dtype):
    import torch
    rng = np.random.default_rng(T * D + ps)
    P = -(-T // ps) + 3
    slots = rng.permutation(P * ps)[:T].astype(np.int32)
    slots[rng.uniform(size=T) < 0.1] = -1
    wide = _rows(rng, (T, 3 * Hkv, D), dtype)
    k, v = wide[:, Hkv:2 * Hkv], wide[:, 2 * Hkv:]  # slices of a projection
    kv = torch.randint(0, 256, (P, Hkv, 9 * ps * D // 8), dtype=torch.uint8, device="cuda")
    want = kv.cpu().numpy().copy()
    pa.paged_attn_append_kv4(k, v, _t(slots), kv)
    R.write(want, slots, _np(k), _np(v), ps)
    np.testing.assert_array_equal(kv.cpu().numpy(), want)
    got_k, got_v = (torch.full((T, Hkv, D), 7.0, dtype=_dt(dtype), device="cuda") for _ in "kv")
    pa.paged_attn_gather_kv4(kv, _t(slots), got_k, got_v)
    for got, x in zip((got_k, got_v), R.values(want, ps, D)):
        held = x.transpose(0, 2, 1, 3).reshape(P * ps, Hkv, D)[np.maximum(slots, 0)]
        np.testing.assert_array_equal(_np(got), np.where(slots[:, None, None] >= 0, held, 0.0))
    assert pa.paged_attn_last_error_word() == 0


def test_rows_all_scales(pa):
    """Every scale, and on either side of every border between two of them."""
    import torch
    mid = 7 * (R.SCALES[:-1] + R.SCALES[1:]) / 2
    tops = np.concatenate([7 * R.SCALES, mid, np.nextafter(np.float32(mid), 0), np.nextafter(np.float32(mid), 9e9),
                           [7 * 7200, 1e30, 3.4e38, 1e-38, 1e-45]]).astype(np.float32)
    T = len(tops)
    x = np.zeros((T, 1, 64), np.float32)
    x[:, 0] = np.random.default_rng(5).uniform(-1, 1, (T, 64)).astype(np.float32) * tops[:, None]
    x[:, 0, ::16] = tops[:, None]
    for side in (1, -1):
        kv = pa.kv4_pool(-(-T // 16), 16, 1, 64)
        want = kv.cpu().numpy()
        slots = np.arange(T, dtype=np.int32)
        pa.paged_attn_append_kv4(_t(side * x), _t(-side * x), _t(slots), kv)
        R.write(want, slots, side * x.astype(np.float64), -side * x.astype(np.float64), 16)
        np.testing.assert_array_equal(kv.cpu().numpy(), want)
    assert pa.paged_attn_last_error_word() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_not_finite(pa, dtype):
    """NaN counts as 0, infinities as the largest value; both are reported, and nothing else changes."""
    import torch
    rng = np.random.default_rng(3)
    for bad in (np.nan, np.inf, -np.inf):
        k, v = _rows(rng, (20, 2, 64), dtype), _rows(rng, (20, 2, 64), dtype)
        k[7, 1, 30], v[9, 0, 2] = bad, bad
        kv = pa.kv4_pool(2, 16, 2, 64)
        want = kv.cpu().numpy()
        slots = np.arange(20, dtype=np.int32)
        pa.paged_attn_append_kv4(k, v, _t(slots), kv)
        R.write(want, slots, _np(k), _np(v), 16)
        np.testing.assert_array_equal(kv.cpu().numpy(), want)
        assert pa.paged_attn_last_error_status() == (pa.PA_OK, pa.ERRBIT_NONFINITE)
    # in a row that is not written nothing is reported
    slots[:] = -1
    pa.paged_attn_append_kv4(k, v, _t(slots), kv)
    assert pa.paged_attn_last_error_word() == 0


def test_rows_bad_slots(pa):
    import torch
    rng = np.random.default_rng(4)
    k, v = _rows(rng, (6, 2, 128), "bf16"), _rows(rng, (6, 2, 128), "bf16")
    kv = torch.randint(0, 256, (3, 2, 9 * 16 * 16), dtype=torch.uint8, device="cuda")
    want = kv.cpu().numpy().copy()
    slots = np.array([48, -2, 5, 2**31 - 1, -2**31, -1], np.int32)
    pa.paged_attn_append_kv4(k, v, _t(slots), kv)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE
    R.write(want, slots, _np(k), _np(v), 16)
    np.testing.assert_array_equal(kv.cpu().numpy(), want)
    a, b = torch.ones_like(k), torch.ones_like(v)
    pa.paged_attn_gather_kv4(kv, _t(slots), a, b)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE
    assert not _np(a)[[0, 1, 3, 4, 5]].any() and _np(a)[2].any() and not _np(b)[[0, 1, 3, 4, 5]].any()


# ----------------------------------------------------------------------------- attention
def _case(seed, lens, new, Hkv, G, D, ps, dtype, pads=0, spare=2, width=None):
    """A pool of random rows with garbage behind the last keys, shuffled pages, ragged packed queries."""
    import torch
    rng = np.random.default_rng(seed)
    lens, new = np.asarray(lens), np.asarray(new)
    need = -(-lens // ps)
    P = int(need.sum()) + spare
    pool = rng.integers(0, 256, (P, Hkv, 9 * ps * D // 8)).astype(np.uint8)
    ids = rng.permutation(P).astype(np.int32)
    W = width or int(need.max()) + 1
    table = np.full((len(lens), W), 0x7FFFFFFF, np.int32)
    table[np.arange(W)[None] < need[:, None]] = ids[:int(need.sum())]
    slots = np.concatenate([table[b, np.arange(n) // ps] * ps + np.arange(n) % ps for b, n in enumerate(lens)] + [[]])
    rows = rng.standard_normal((2, len(slots), Hkv, D)) * (1 + 2 * (np.arange(D) % 37 == 5))
    R.write(pool, slots, rows[0], rows[1], ps)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((starts[-1] + pads, Hkv * G, D))).to(_dt(dtype)).cuda()
    return dict(q=q, kv=_t(pool), pool=pool, ps=ps, table=table, lens=lens.astype(np.int32), starts=starts, dtype=dtype)


def _check(pa, c, causal=True, q_offset=None, scale=None, packed=True, q=None, err=0, workspace=None):
    import torch
    q = c["q"] if q is None else q
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T, Hq, D), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T, Hq), 5.0, device="cuda")
    qo = None if q_offset is None else _t(q_offset, np.int32)
    if packed:
        pa.paged_attn_fwd_kv4(q, c["kv"], _t(c["table"]), _t(c["lens"]), causal, qo, scale, out, lse,
                              q_start=_t(c["starts"]), workspace=workspace)
    else:
        B = len(c["lens"])
        pa.paged_attn_fwd_kv4(q.view(B, -1, Hq, D), c["kv"], _t(c["table"]), _t(c["lens"]), causal, qo, scale,
                              out.view(B, -1, Hq, D), lse.view(B, -1, Hq), workspace=workspace)
    assert pa.paged_attn_last_error_word() == err
    told = (causal, scale, None if q_offset is None else tuple(q_offset), c["table"].tobytes())
    if told not in c:  # the same rows are checked with several workspaces
        c[told] = R.attention(_np(q), c["pool"], c["ps"], c["table"], c["lens"], c["starts"], causal, q_offset, scale)
    want, want_lse, off, room, mass = c[told]
    got, got_lse = _np(out), _np(lse)
    own = ~np.isnan(want_lse)
    assert (got[~own] == 5.0).all() and (got_lse[~own] == 5.0).all()  # rows of no sequence
    empty = own & np.isneginf(want_lse)
    assert (got[empty] == 0).all() and np.isneginf(got_lse[empty]).all()
    own &= ~empty
    bar = STEP[c["dtype"]] * np.abs(want) + room + WEIGHT[c["dtype"]] * mass + 2.0 ** -24
    worst = np.abs(got - want)[own] / bar[own]
    assert worst.size == 0 or worst.max() <= 1, f"output off by {worst.max():.3g} of its bar"
    worst = np.abs(got_lse[own] - want_lse[own]) / (off + 2.0 ** -22 * np.abs(want_lse))[own]
    assert worst.size == 0 or worst.max() <= 1, f"lse off by {worst.max():.3g} of its bar"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ps", [16, 32, 64])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 8, 12, 16, 24, 40])
def test_decode(pa, G, D, ps, dtype):
    c = _case(G * D + ps, [1, 15, 16, 17, 63, 64, 65, 200, 129], [1] * 9, 2, G, D, ps, dtype)
    _check(pa, c)


@pytest.mark.parametrize("D,G,dtype", [(64, 3, "f16"), (128, 4, "bf16"), (128, 16, "f16"), (256, 2, "bf16")])
@pytest.mark.parametrize("causal", [False, True])
def test_ragged_runs(pa, D, G, dtype, causal):
    """Runs of 0 to 40 tokens beside single ones, sequences without keys, rows behind the last one."""
    c = _case(D + G, [0, 70, 33, 5, 300, 64, 0, 18], [3, 40, 1, 5, 2, 17, 0, 18], 3, G, D, 16, dtype, pads=6)
    _check(pa, c, causal)


@pytest.mark.parametrize("causal", [False, True])
def test_uniform_and_offsets(pa, causal):
    c = _case(8, [40, 90, 7, 64], [6] * 4, 2, 4, 128, 32, "bf16")
    _check(pa, c, causal, packed=False)
    # the first tokens see nothing, some only a part, some past the end
    _check(pa, c, causal, q_offset=[-9, 3, 100, -3], packed=False)
    _check(pa, c, causal, q_offset=[-9, 3, 100, -3])


RUNS = [([1500, 900], [300, 200], 2, 8, 128, 16, "bf16"), ([1100, 700, 130], [129, 64, 130], 2, 4, 128, 64, "f16"),
        ([2000, 64, 9, 800], [500, 64, 1, 33], 3, 3, 64, 32, "bf16"), ([1000], [257], 1, 24, 64, 16, "f16"),
        ([700, 300], [70, 90], 1, 100, 128, 16, "bf16"), ([2100, 1800, 5, 900], [700, 1, 5, 300], 2, 1, 128, 16, "f16"),
        ([1300, 0, 640], [400, 10, 0], 2, 16, 128, 32, "bf16"),
        # few tiles over many keys: several CTAs share them
        ([7000, 300], [260, 3], 1, 8, 128, 16, "bf16"), ([5000], [200], 1, 12, 128, 32, "f16")]
SHARED = {0, 2, 6, 7, 8}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(RUNS)))
def test_runs(pa, case, causal):
    """Prompt chunks over longer caches (tcgen05), beside single tokens and short runs; rows behind the last
    sequence; tiles that end inside a page and inside a token's heads."""
    import torch
    lens, new, Hkv, G, D, ps, dtype = RUNS[case]
    c = _case(case + 50, lens, new, Hkv, G, D, ps, dtype, pads=5)
    _check(pa, c, causal)
    need = pa.paged_attn_kv4_workspace_bytes(len(lens), c["q"].shape[0], Hkv * G, Hkv, D, ps, c["table"].shape[1],
                                             torch.cuda.get_device_properties(0).multi_processor_count, pa.PA_BF16)
    assert (need > 0) == (case in SHARED)
    if need:
        _check(pa, c, causal, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
        _check(pa, c, causal, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("case", [(128, 8, "bf16"), (64, 4, "f16")])
def test_uniform_runs(pa, case):
    """Also with tokens that see nothing, a part, or past the end; a negative scale, none, and scores in the thousands;
    pages outside the pool; strided queries."""
    import torch
    D, G, dtype = case
    c = _case(D, [900, 1200], [200, 200], 2, G, D, 16, dtype)
    _check(pa, c, packed=False)
    _check(pa, c, q_offset=[-70, 1100], packed=False)
    for scale in (-0.4, 0.0, 30.0):
        _check(pa, c, scale=scale, packed=False)
    T, Hq, _ = c["q"].shape
    wide = torch.randn((T, Hq + 4, D), device="cuda").to(c["q"].dtype)
    wide[:, :Hq] = c["q"]
    _check(pa, c, q=wide[:, :Hq])
    c["table"][0, 3], c["table"][1, 70] = -1, 10**8
    _check(pa, c, packed=False, err=pa.ERRBIT_PAGE_RANGE)


LONG = [([9000], [1], 1, 4, 128, 16, "bf16"), ([5000, 33], [2, 1], 2, 8, 64, 64, "f16"), ([3000], [1], 1, 2, 256, 32, "bf16"),
        ([100], [1], 1, 4, 128, 16, "bf16"), ([20000, 0, 700], [3, 1, 0], 1, 8, 128, 32, "f16")]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_few_rows_many_keys(pa, case):
    """Few rows over many pages: with a workspace the whole grid shares the keys, without one clusters do; both beside
    sequences that leave most of their CTAs without keys, and in a table far wider than any sequence."""
    import torch
    lens, new, Hkv, G, D, ps, dtype = LONG[case]
    c = _case(case, lens, new, Hkv, G, D, ps, dtype, pads=2, width=1400)
    need = pa.paged_attn_kv4_workspace_bytes(len(lens), c["q"].shape[0], Hkv * G, Hkv, D, ps, 1400,
                                             torch.cuda.get_device_properties(0).multi_processor_count, pa.PA_BF16)
    assert need > 0
    _check(pa, c)
    _check(pa, c, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    for less in (0, need - 1):
        _check(pa, c, workspace=torch.empty(less, dtype=torch.uint8, device="cuda"))
    c["table"][0, 1] = -1
    _check(pa, c, causal=False, err=pa.ERRBIT_PAGE_RANGE)


MANY = [  # sequences, kv heads, G, head_dim, new tokens of each (None: one, but for two that share theirs out), all one length
    (256, 4, 2, 64, 1, False), (130, 5, 4, 64, 1, True), (200, 4, 1, 128, None, False), (60, 4, 4, 64, 9, False), (33, 19, 3, 256, 1, False)]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_more_sequences_than_fit_at_once(pa, case):
    """Batches of several waves, whose longest sequences are taken first: lengths of all sizes, none among them, and all
    alike."""
    B, Hkv, G, D, new, same = MANY[case]
    rng = np.random.default_rng(80 + case)
    lens = np.full(B, 40) if same else np.where(rng.uniform(size=B) < 0.8, rng.integers(0, 120, B), rng.integers(100, 900, B))
    if not same:
        lens[rng.integers(0, B)] = 2080
    count = np.full(B, new or 1)
    if new is None:
        count[7], count[B - 1] = 2, 0
    c = _case(90 + case, lens, count, Hkv, G, D, 16, "bf16", width=130)
    _check(pa, c, packed=new in (None, 1))


def test_many_single_tokens_beside_runs(pa):
    """Both kernels at once, the second over the short runs of a batch of several waves."""
    rng = np.random.default_rng(99)
    B = 130
    new = np.where(np.arange(B) % 40 == 7, 200, rng.integers(0, 4, B))
    lens = np.where(new == 200, 400, rng.integers(0, 200, B))
    lens[3] = 2080
    lens = np.maximum(lens, new)
    _check(pa, _case(99, lens, new, 4, 8, 64, 16, "bf16", pads=3, width=130))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5, 40.0])
def test_scales(pa, scale):
    """Also scores up to thousands: one key takes everything, references move far."""
    _check(pa, _case(12, [150, 31], [3, 1], 2, 4, 128, 16, "bf16"), scale=scale)


@pytest.mark.parametrize("D,dtype", [(64, "f16"), (128, "bf16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("low,high,scale", [(0, 8, 1000.0), (1, 3, -4000.0), (0xD0, 0x100, 1e-5)])
def test_smallest_and_largest_scales(pa, low, high, scale, D, dtype):
    """Scale bytes below the normal numbers and around the largest, single tokens and a run beside them."""
    c = _case(95 + low, [300, 90, 17, 0], [70, 1, 2, 1], 2, 4, D, 16, dtype)
    c["pool"][:, :, 16 * D:] = np.random.default_rng(low).integers(low, high, c["pool"][:, :, 16 * D:].shape)
    c["kv"] = _t(c["pool"])
    _check(pa, c, scale=scale)


def test_strided_queries(pa):
    import torch
    c = _case(13, [80, 40], [5, 2], 2, 4, 128, 16, "bf16")
    T, Hq, D = c["q"].shape
    wide = torch.randn((T, Hq + 4, D), device="cuda").bfloat16()
    wide[:, :Hq] = c["q"]
    _check(pa, c, q=wide[:, :Hq])


def test_bad_pages(pa):
    """Ids outside the pool read as zeros; other sequences do not notice."""
    c = _case(14, [100, 70, 200], [2, 1, 1], 2, 4, 128, 16, "bf16")
    c["table"][0, 2], c["table"][1, 0], c["table"][2, 12] = -1, c["pool"].shape[0], -2**31
    _check(pa, c, err=pa.ERRBIT_PAGE_RANGE)


def test_clipped_lengths(pa):
    c = _case(15, [64, 40], [1, 1], 1, 2, 64, 16, "f16", width=4)
    c["lens"][0] = 1000  # more than the row's four pages
    _check(pa, c, err=pa.ERRBIT_SEQ_CLIPPED)


def test_malformed_ranges(pa):
    """Entries of q_start outside the rows or decreasing: their sequences are skipped and reported."""
    import torch
    c = _case(16, [64, 40, 50], [2, 3, 2], 1, 2, 64, 16, "f16")
    for starts in ([0, 2, 9, 7], [-1, 2, 5, 7], [0, 5, 2, 7], [3, 2, 5, 100]):
        out = torch.full_like(c["q"], 5.0)
        pa.paged_attn_fwd_kv4(c["q"], c["kv"], _t(c["table"]), _t(c["lens"]), True, None, 0.1, out, None,
                              q_start=_t(starts, np.int32))
        assert pa.paged_attn_last_error_status() == (pa.PA_EINVAL, pa.ERRBIT_QSTART)


def test_convenience_and_graph(pa):
    """Captured append and attention, replayed on new contents; another stream."""
    import torch
    c = _case(17, [48, 20], [1, 1], 2, 4, 128, 16, "bf16")
    kv, table, lens, starts = c["kv"], _t(c["table"]), _t(c["lens"]), _t(c["starts"])
    ref, ref_lse = pa.attention_kv4(c["q"], kv, table, lens, q_start=starts, want_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pa.attention_kv4(c["q"], kv, table, lens, q_start=starts, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    k = torch.randn((2, 2, 128), device="cuda").bfloat16()
    slots = _t([c["table"][0, 2] * 16 + 15, c["table"][1, 1] * 16 + 3], np.int32)
    out = torch.empty_like(c["q"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.paged_attn_append_kv4(k, k, slots, kv)
        pa.paged_attn_fwd_kv4(c["q"], kv, table, lens, True, None, 128 ** -0.5, out, None, q_start=starts)
    for seed in range(2):
        k.copy_(torch.randn((2, 2, 128), generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        got = out.clone()
        pa.paged_attn_append_kv4(k, k, slots, kv)
        assert torch.equal(got, pa.attention_kv4(c["q"], kv, table, lens, q_start=starts))
    assert pa.paged_attn_last_error_word() == 0


def test_pool_past_four_gibibytes(pa):
    """Pages whose bytes lie past 2^32: written, read back and attended to by both kernels."""
    import torch
    ps, Hkv, G, D, P = 64, 8, 4, 128, 64000
    kv = pa.kv4_pool(P, ps, Hkv, D)
    assert kv.numel() > 1.08 * 2**32
    lens, new = np.array([70, 3000]), np.array([1, 300])
    need = -(-lens // ps)
    table = np.full((2, int(need.max())), -1, np.int32)
    ids = np.r_[np.arange(P - 40, P), np.arange(10)][::-1]
    table[0, :need[0]], table[1, :need[1]] = ids[:need[0]], ids[need[0]:need.sum()]
    pos = [np.arange(n) for n in lens]
    slots = np.concatenate([table[b, p // ps] * np.int64(ps) + p % ps for b, p in enumerate(pos)])
    k, v = (torch.randn((len(slots), Hkv, D), device="cuda").bfloat16() for _ in "kv")
    pa.paged_attn_append_kv4(k, v, _t(slots, np.int32), kv)
    a, b = torch.empty_like(k), torch.empty_like(v)
    pa.paged_attn_gather_kv4(kv, _t(slots, np.int32), a, b)
    # the same sequences in a small pool
    used = np.unique(table[table >= 0])
    pool = kv[torch.from_numpy(used.astype(np.int64)).cuda()].cpu().numpy()
    small = np.where(table >= 0, np.searchsorted(used, np.maximum(table, 0)), -1).astype(np.int32)
    for got, want in zip((a, b), R.values(pool, ps, D)):
        flat = want.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
        at = np.concatenate([small[i, p // ps] * ps + p % ps for i, p in enumerate(pos)])
        np.testing.assert_array_equal(_np(got), flat[at])
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn((starts[-1], Hkv * G, D), device="cuda").bfloat16()
    out = pa.attention_kv4(q, kv, _t(table), _t(lens, np.int32), q_start=_t(starts))
    near = pa.attention_kv4(q, _t(pool), _t(small), _t(lens, np.int32), q_start=_t(starts))
    assert torch.equal(out, near)
    rows = np.r_[0, 1, 150, 300]
    want, _, _, room, mass = R.attention(_np(q[:1]), pool, ps, small[:1], lens[:1], [0, 1], True, None, D ** -0.5)
    assert (np.abs(_np(out[:1]) - want) <= STEP["bf16"] * np.abs(want) + room + WEIGHT["bf16"] * mass).all()
    for t in rows[1:]:
        n = int(lens[1] - new[1] + t)  # keys of the token
        want, _, _, room, mass = R.attention(_np(q[t:t + 1]), pool, ps, small[1:], [n], [0, 1], True, None, D ** -0.5)
        assert (np.abs(_np(out[t:t + 1]) - want) <= STEP["bf16"] * np.abs(want) + room + WEIGHT["bf16"] * mass).all()
    assert pa.paged_attn_last_error_word() == 0


def test_two_streams_at_once(pa):
    """Calls that share their keys out, side by side on two streams, each with a workspace of its own; one captured
    and replayed on a stream of its own beside an eager one."""
    import torch
    cases = [_case(30 + i, [6000 - 900 * i], [2], 1, 4, 128, 16, "bf16", width=600) for i in range(2)]
    args = [(c["q"], c["kv"], _t(c["table"]), _t(c["lens"])) for c in cases]
    starts = [_t(c["starts"]) for c in cases]
    want = [pa.attention_kv4(*a, q_start=s) for a, s in zip(args, starts)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(pa.attention_kv4(*args[i], q_start=starts[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = pa.attention_kv4(*args[0], q_start=starts[0])
    for _ in range(5):
        kept.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            other = pa.attention_kv4(*args[1], q_start=starts[1])
        torch.cuda.synchronize()
        assert torch.equal(kept, want[0]) and torch.equal(other, want[1])


def test_memory_of_another_stream(pa):
    """What a call on another stream allocates is not memory that the current stream's pending work may still use."""
    import torch
    c = _case(60, [6000], [2], 1, 4, 128, 16, "bf16", width=600)
    args, starts = (c["q"], c["kv"], _t(c["table"]), _t(c["lens"])), _t(c["starts"])
    want, want_lse = pa.attention_kv4(*args, q_start=starts, want_lse=True)
    size = pa.paged_attn_kv4_workspace_bytes(1, 2, 4, 1, 128, 16, 600, torch.cuda.get_device_properties(0).multi_processor_count)
    assert size > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(want), torch.empty_like(want_lse), torch.empty(size, dtype=torch.uint8, device="cuda")]
    freed = {t.data_ptr() for t in freed}  # and given back
    out, lse = pa.attention_kv4(*args, q_start=starts, want_lse=True, stream=side)
    assert out.data_ptr() not in freed and lse.data_ptr() not in freed
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("tokens,Hkv", [(1, 1), (16, 16)])
def test_nearly_two_to_the_31_keys(pa, tokens, Hkv):
    """The longest sequence that there can be.  All but its last five pages are one page whose keys weigh nothing."""
    import torch
    ps, G, D = 64, 8, 64
    rng = np.random.default_rng(70)
    pool = np.zeros((4, Hkv, 9 * ps * D // 8), np.uint8)
    rows = rng.standard_normal((2, 4 * ps, Hkv, D))
    rows[0, :, :, :16] = 0
    rows[0, :ps, :, :16] = -7.0
    R.write(pool, np.arange(4 * ps), rows[0], rows[1], ps)
    q = rng.standard_normal((tokens, Hkv * G, D))
    q[:, :, :16] = 8.0  # with the weightless page: a score some 100 below the others'
    q = torch.from_numpy(q).bfloat16().cuda()
    W = 2**25 - 1
    table = torch.zeros((1, W), dtype=torch.int32, device="cuda")
    table[0, -5:] = torch.tensor([1, 2, 3, 1, 2], device="cuda")
    lens = _t([W * ps], np.int32)
    out = pa.attention_kv4(q[None], _t(pool), table, lens)[0]
    assert pa.paged_attn_last_error_word() == 0
    want, _, _, room, mass = R.attention(_np(q), pool, ps, np.array([[0, 1, 2, 3, 1, 2]], np.int32), np.array([6 * ps], np.int32),
                                         [0, tokens], True, None, D ** -0.5)
    assert (np.abs(_np(out) - want) <= STEP["bf16"] * np.abs(want) + room + WEIGHT["bf16"] * mass + 2.0 ** -24).all()
