"""The serving step over selected pages on the GPU: tables and slots, append with page envelopes, page
selection and attention over the selected pages, each against the plain implementation
(tests/_sparse_ref.py), then run together.

What the calls compute in whole numbers or exactly (tables, slots, cache rows, envelopes, selections)
must match bit for bit.  Attention is held to the library's bars: half a rounding step of the output
type (bf16 2^-8, f16 2^-11 relative, within rtol 2^-8) on top of the float32 sums, whose error at unit
normal inputs is at most 2 max|v| D 2^-24 sum|q_d k_d| scale = 2 * 4 * 256 * 2^-24 * 16 < 2e-3.
"""
import numpy as np
import pytest

from paged_kv_cache_201_gb300 import workloads as W
from tests import _gpu
from tests import _sparse_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_201_gb300 as pa
    pa.load_library(build_if_missing=True)
    pa.paged_attn_last_error_word()
    return pa


def _t(a, dtype=None):
    import torch
    x = torch.from_numpy(np.ascontiguousarray(a, dtype=dtype))
    return x.cuda()


def _bits(t, dtype):
    return _gpu.to_host_elems(t, dtype)


def _raw(a):
    a = np.ascontiguousarray(a)
    return a.view(np.uint32) if a.dtype == np.float32 else a


# ----------------------------------------------------------------------------- tables and slots
def _run_tables(pa, cached, new, free, count, table, total, ps, num_pages, alias=False):
    import torch
    B = len(cached)
    c, n, f, cnt, bt = _t(cached, np.int32), _t(new, np.int32), _t(free, np.int32), _t([count], np.int32), _t(table)
    sl = c if alias else torch.full((B,), -7, dtype=torch.int32, device="cuda")
    left = cnt if alias else torch.full((1,), -7, dtype=torch.int32, device="cuda")
    qo, qs = torch.full((B,), -7, dtype=torch.int32, device="cuda"), torch.full((B + 1,), -7, dtype=torch.int32,
                                                                               device="cuda")
    slots = torch.full((total,), -7, dtype=torch.int32, device="cuda")
    pa.paged_attn_step_tables(c, n, f, cnt, bt, sl, qo, qs, slots, left, ps, num_pages)
    bits = pa.paged_attn_last_error_word()
    return {"table": bt.cpu().numpy(), "seq_lens": sl.cpu().numpy(), "q_offset": qo.cpu().numpy(),
            "q_start": qs.cpu().numpy(), "slots": slots.cpu().numpy(), "free_left": left.cpu().numpy()}, bits


def _check_tables(pa, cached, new, free, count, table, total, ps, num_pages, alias=False):
    want = R.step_tables(np.asarray(cached), np.asarray(new), free, count, table, total, ps, num_pages)
    got, bits = _run_tables(pa, cached, new, free, count, table, total, ps, num_pages, alias)
    for k, v in got.items():
        np.testing.assert_array_equal(v, want[k], err_msg=k)
    assert bool(bits & pa.ERRBIT_REFUSED) == want["refused"]
    assert bool(bits & pa.ERRBIT_PAGE_RANGE) == want["bad_page"]
    assert not bits & ~(pa.ERRBIT_REFUSED | pa.ERRBIT_PAGE_RANGE)
    return want


def _tables_case(seed, B, width, ps, chunk, count, idle=0.1):
    rng = np.random.default_rng(seed)
    new = np.where(rng.uniform(size=B) < 0.6, 1, rng.integers(1, chunk + 1, B))
    new[rng.uniform(size=B) < idle] = 0
    cached = np.minimum(rng.integers(0, width * ps, B), np.maximum(width * ps - new, 0))
    cached[rng.uniform(size=B) < 0.2] = 0
    exact = rng.uniform(size=B) < 0.2
    cached[exact] = cached[exact] // ps * ps  # the last page is full
    need = -(-cached // ps)
    pages = int(need.sum()) + count
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), W.SENTINEL_MAX, np.int32)
    table[np.arange(width)[None] < need[:, None]] = ids[:int(need.sum())]
    return cached.astype(np.int32), new.astype(np.int32), ids[int(need.sum()):], table, pages


@pytest.mark.parametrize("ps", [16, 32, 64])
@pytest.mark.parametrize("B,width,chunk", [(1, 4, 1), (1, 40, 600), (33, 20, 50), (1024, 24, 40), (1025, 6, 3),
                                           (5000, 4, 9)])
@pytest.mark.parametrize("alias", [False, True])
def test_tables(pa, B, width, chunk, ps, alias):
    cached, new, free, table, pages = _tables_case(B + ps, B, width, ps, min(chunk, width * ps), B * 3 + 50)
    total = int(new.sum()) + 13
    want = _check_tables(pa, cached, new, free, len(free), table, total, ps, pages, alias)
    assert not want["refused"] and want["q_start"][-1] == new.sum()


def test_tables_largest_batch(pa):
    B = 16384
    cached, new, free, table, pages = _tables_case(3, B, 3, 16, 5, 3 * B)
    _check_tables(pa, cached, new, free, len(free), table, int(new.sum()), 16, pages)


@pytest.mark.parametrize("count,total", [(7, 4000), (4000, 61), (0, 300), (9, 100)])
def test_tables_too_few_pages_or_slots(pa, count, total):
    """Requests past the free pages or the slots are turned down; those that need no page and fit go on."""
    cached, new, free, table, pages = _tables_case(11, 60, 20, 16, 40, 4000)
    want = _check_tables(pa, cached, new, free, count, table, total, 16, pages)
    assert want["refused"]


def test_tables_odd_requests(pa):
    """Negative lengths, rows without room, a free count past the stack, ids outside the pool, idle
    requests, lengths whose sum passes 31 bits."""
    ps, width = 16, 4
    cached = np.array([-1, 5, 64, 63, 0, 10, 2**31 - 1, 16, 3], np.int32)
    new = np.array([3, -2, 1, 1, 65, 0, 2**31 - 1, 16, 0], np.int32)
    table = np.arange(9 * width, dtype=np.int32).reshape(9, width)
    table[3, 3] = -5  # the last token of request 3 lands in a page outside the pool
    free = np.array([50, 99, 1], np.int32)  # 99 is outside it too
    _check_tables(pa, cached, new, free, 3, table, 100, ps, 60)
    _check_tables(pa, cached, new, free, 2, table, 100, ps, 60)
    _check_tables(pa, cached, new, free, 8, table, 100, ps, 60)
    _check_tables(pa, cached, new, free, -3, table, 100, ps, 60)
    _check_tables(pa, np.zeros(4, np.int32), np.zeros(4, np.int32), free, 3, table[:4], 0, ps, 60)


# ----------------------------------------------------------------------------- append
def _append_case(seed, q_lens, seq_lens, Hkv, D, ps, dtype, pads=3):
    b = R.Batch(seed, q_lens, seq_lens, Hkv, Hkv, D, ps, dtype)
    rng = np.random.default_rng(seed + 1)
    slots = []
    for s, n in enumerate(q_lens):
        for x in range(int(b.seq_lens[s]) - n, int(b.seq_lens[s])):
            slots.append(int(b.table[s, x // ps]) * ps + x % ps)
    slots += [-1] * pads
    shape = (len(slots), Hkv, D)
    return b, np.asarray(slots, np.int32), R.random_elems(rng, shape, dtype), R.random_elems(rng, shape, dtype)


def _run_append(pa, b, slots, kn, vn, env=True, strided=False):
    import torch
    dt = b.dtype
    d = b.device()
    kd, vd = W.host_to_torch(kn, dt).cuda(), W.host_to_torch(vn, dt).cuda()
    if strided:  # slices of one projection's output, other elements NaN
        T, Hkv, D = kn.shape
        fused = torch.full((T, 3 * Hkv, D), float("nan"), dtype=kd.dtype, device="cuda")
        fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:] = kd, vd
        kd, vd = fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:]
    e = s = None
    if env:
        e = torch.full((b.P, b.Hkv, 2, b.D), 77, dtype=torch.int8, device="cuda")
        s = torch.full((b.P, b.Hkv), -1.0, device="cuda")
    pa.paged_attn_append(kd, vd, _t(slots), d["k"], d["v"], e, s)
    torch.cuda.synchronize()
    return (_bits(d["k"], dt), _bits(d["v"], dt), None if e is None else e.cpu().numpy(),
            None if s is None else s.cpu().numpy())


def _check_append(pa, b, slots, kn, vn, env=True, strided=False):
    k, v = b.k.copy(), b.v.copy()
    e = np.full((b.P, b.Hkv, 2, b.D), 77, np.int8) if env else None
    s = np.full((b.P, b.Hkv), -1.0, np.float32) if env else None
    R.append(kn, vn, slots, k, v, b.dtype, e, s)
    gk, gv, ge, gs = _run_append(pa, b, slots, kn, vn, env, strided)
    np.testing.assert_array_equal(_raw(gk), _raw(k))
    np.testing.assert_array_equal(_raw(gv), _raw(v))
    if env:
        np.testing.assert_array_equal(gs, s)
        np.testing.assert_array_equal(ge, e)


APPEND_BATCHES = [([1], [1]), ([1, 1, 1], [16, 17, 64]), ([5, 1, 130, 16, 0], [5, 40, 131, 32, 9]),
                  ([200], [333])]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hkv,D,ps", [(1, 64, 16), (3, 128, 32), (8, 128, 16), (2, 256, 64), (5, 64, 64)])
@pytest.mark.parametrize("q_lens,seq_lens", APPEND_BATCHES)
def test_append(pa, dtype, Hkv, D, ps, q_lens, seq_lens):
    b, slots, kn, vn = _append_case(D + ps, q_lens, seq_lens, Hkv, D, ps, dtype)
    _check_append(pa, b, slots, kn, vn, strided=len(q_lens) > 1)


@pytest.mark.parametrize("dtype,D,ps", [("bf16", 64, 16), ("f16", 128, 64), ("f32", 64, 32), ("bf16", 256, 16)])
def test_append_many_tokens(pa, dtype, D, ps):
    """Enough tokens for several to a warp; the last warp holds fewer."""
    b, slots, kn, vn = _append_case(D + ps, [1900, 1, 0, 3, 149], [1913, 77, 5, 3, 160], 8, D, ps, dtype, pads=1)
    assert len(slots) * 8 >= 16384 and len(slots) % 4
    slots[700:703] = -1  # a hole: its page ends before it and goes on behind it
    slots[703:720] = -1
    _check_append(pa, b, slots, kn, vn, strided=True)


def test_append_without_envelopes_any_order(pa):
    """Without envelopes the tokens may come in any order."""
    b, slots, kn, vn = _append_case(4, [9, 40], [50, 40], 2, 128, 16, "bf16")
    perm = np.random.default_rng(0).permutation(len(slots))
    _check_append(pa, b, slots[perm], kn[perm], vn[perm], env=False)


def test_append_token_by_token_gives_the_same_envelopes(pa):
    import torch
    b, slots, kn, vn = _append_case(5, [37], [37], 2, 128, 32, "bf16", pads=0)
    _, _, e, s = _run_append(pa, b, slots, kn, vn)
    d = b.device()
    env, scale = torch.full((b.P, 2, 2, 128), 77, dtype=torch.int8, device="cuda"), torch.full((b.P, 2), -1.0,
                                                                                            device="cuda")
    kd, vd, sd = W.host_to_torch(kn, "bf16").cuda(), W.host_to_torch(vn, "bf16").cuda(), _t(slots)
    for t in range(37):
        pa.paged_attn_append(kd[t:t + 1], vd[t:t + 1], sd[t:t + 1], d["k"], d["v"], env, scale)
    np.testing.assert_array_equal(env.cpu().numpy(), e)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_special_values(pa, dtype):
    """NaN and infinite keys mark the page; zero keys, the smallest and the largest numbers quantise."""
    b, slots, kn, vn = _append_case(6, [16] * 6, [16] * 6, 2, 64, 16, dtype, pads=0)
    f32 = dtype == "f32"
    one = lambda x: np.float32(x) if f32 else W.bf16_bits_rne(np.float32([x]))[0]  # noqa: E731
    kn[3, 0, 7] = one(np.nan)
    kn[16 + 5, 1, 9] = one(-np.inf)
    kn[32:48] = one(0.0)
    kn[48:64] = one(0.0)
    kn[50, 0, 3] = one(1e-39)  # below the smallest normal number
    kn[64:80, 0] = one(3e38)
    kn[66, 0, 1] = one(-3.3e38)
    _check_append(pa, b, slots, kn, vn)


def test_append_bad_slots(pa):
    """Slots outside the pool are skipped and reported; -1 is skipped in silence."""
    b, slots, kn, vn = _append_case(7, [6], [20], 2, 128, 16, "f16")
    pa.paged_attn_last_error_word()
    _check_append(pa, b, slots, kn, vn)
    assert pa.paged_attn_last_error_word() == 0
    slots[1], slots[4] = b.P * 16, -9
    b2 = R.Batch(7, [6], [20], 2, 2, 128, 16, "f16")
    _check_append(pa, b2, slots, kn, vn, env=False)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE


# ----------------------------------------------------------------------------- selection
def _run_select(pa, b, env, scale, sink, local, K, causal=True, q_offset=None, uniform=False, q=None):
    import torch
    d = b.device()
    q = d["q"] if q is None else q
    qo = None if q_offset is None else _t(q_offset, np.int32)
    sel = torch.full((q.shape[0], b.Hkv, K), -9, dtype=torch.int32, device="cuda")
    if uniform:
        B = len(b.q_lens)
        pa.paged_attn_select_pages(q.view(B, -1, b.Hq, b.D), _t(env), _t(scale), d["table"], d["lens"], causal, qo,
                                   sink, local, sel.view(B, -1, b.Hkv, K), b.ps)
    else:
        pa.paged_attn_select_pages(q, _t(env), _t(scale), d["table"], d["lens"], causal, qo, sink, local, sel, b.ps,
                                   q_start=d["q_start"])
    torch.cuda.synchronize()
    return sel.cpu().numpy()


def _check_select(pa, b, sink, local, K, causal=True, q_offset=None, env=None, uniform=False):
    env = b.envelopes() if env is None else env
    want = R.select(b.q64(), *env, b.table, b.rows(causal, q_offset), b.Hkv, b.ps, sink, local, K)
    got = _run_select(pa, b, *env, sink, local, K, causal, q_offset, uniform)
    np.testing.assert_array_equal(got[:b.T], want)
    assert (got[b.T:] == -9).all()  # rows of no sequence are left as they were
    assert pa.paged_attn_last_error_word() == 0
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 16), (3, 3, 64, 32), (14, 2, 256, 16), (24, 1, 128, 64),
                                         (40, 1, 64, 16), (130, 1, 64, 16)])
def test_select(pa, dtype, Hq, Hkv, D, ps):
    b = R.Batch(Hq + D, [1, 3, 0, 1, 7], [1, 40 * ps, 9, 31 * ps + 5, 23 * ps + 1], Hq, Hkv, D, ps, dtype, q_pad=2)
    for sink, local, K in [(1, 2, 8), (0, 0, 1), (0, 0, 5), (2, 3, 5), (0, 4, 23), (1, 0, 64)]:
        _check_select(pa, b, sink, local, K)


def test_select_masks(pa):
    """Non-causal, explicit offsets (one puts every key out of reach), the uniform layout, a view of q."""
    import torch
    b = R.Batch(2, [4, 4, 4], [900, 30, 500], 8, 2, 128, 16, "bf16")
    _check_select(pa, b, 1, 2, 6, causal=False)
    _check_select(pa, b, 1, 2, 6, q_offset=[300, -9, 496])
    _check_select(pa, b, 1, 2, 6, uniform=True)
    env = b.envelopes()
    fused = torch.full((b.T, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = b.device()["q"]
    got = _run_select(pa, b, *env, 1, 2, 6, q=fused[:, 2:10])
    np.testing.assert_array_equal(got, R.select(b.q64(), *env, b.table, b.rows(), 2, 16, 1, 2, 6))


def test_select_ties_and_marks(pa):
    """Equal scores go to the lowest pages; marked (non-finite) pages come first; a non-finite or zero
    query scores 0 everywhere."""
    b = R.Batch(3, [1, 1, 2], [1600, 1000, 700], 4, 2, 64, 16, "f32")
    env, scale = b.envelopes()
    same = np.broadcast_to(env[:1, :1], env.shape).copy()
    _check_select(pa, b, 1, 1, 9, env=(same, np.ones_like(scale)))
    marked = scale.copy()
    marked[np.random.default_rng(0).uniform(size=scale.shape) < 0.1] = np.inf
    _check_select(pa, b, 1, 1, 9, env=(env, marked))
    _check_select(pa, b, 0, 0, 30, env=(env, np.where(np.isnan(scale), scale, np.float32(3e38))))  # scores overflow
    b.q[0] = 0
    b.q[1, 1, 5] = np.nan
    b.q[2, 3, 0] = np.inf
    _check_select(pa, b, 0, 1, 9)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_select_largest_scores(pa, D):
    """Scores of the largest magnitude that differ by one: every product 127 * 127 or 127 * -127, one
    corner off by one, in both signs."""
    b = R.Batch(D, [1, 1], [200 * 16, 150 * 16], 16, 2, D, 16, "bf16")
    rng = np.random.default_rng(D)
    sign = rng.choice([-1, 1], D)
    b.q[:] = W.bf16_bits_rne(np.broadcast_to(3.0 * sign, b.q.shape).astype(np.float32))
    top = np.where(sign > 0, 127, -127).astype(np.int8)
    env = np.broadcast_to(top, (b.P, b.Hkv, 2, D)).copy()
    env[b.P // 2:] *= -1
    for p in range(b.P):
        d = rng.integers(0, D)
        env[p, :, :, d] -= np.sign(env[p, :, :, d]) * np.int8(rng.integers(0, 3))
    _check_select(pa, b, 1, 1, 30, env=(env, np.ones((b.P, b.Hkv), np.float32)))


@pytest.mark.parametrize("chunk", [64, 300, 700])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2), (8, 2), (8, 1), (32, 8), (12, 1), (32, 1), (40, 1)])
def test_select_prompt_chunks(pa, chunk, Hq, Hkv):
    """Prompt chunks beside single tokens: tokens that share a block, blocks that hold several sequences."""
    b = R.Batch(chunk + Hq, [chunk, 1, 0, 5, 1, 37], [chunk + 600, 900, 3, 5, 700, 200], Hq, Hkv, 64, 16, "bf16",
                q_pad=3)
    _check_select(pa, b, 1, 2, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 16), (3, 1, 128, 32), (2, 2, 64, 64), (14, 2, 128, 16),
                                         (16, 1, 64, 16), (8, 2, 256, 16)])
def test_select_prompt_chunks_types(pa, dtype, Hq, Hkv, D, ps):
    b = R.Batch(Hq + D, [130, 1, 40, 64], [40 * ps + 130, 900, 25 * ps, 64], Hq, Hkv, D, ps, dtype, q_pad=1)
    for sink, local, K in [(1, 2, 8), (0, 0, 1), (2, 3, 5), (0, 0, 23)]:
        _check_select(pa, b, sink, local, K)
    _check_select(pa, b, 1, 2, 6, causal=False)
    _check_select(pa, b, 1, 2, 6, q_offset=[-5, 100, 20 * ps, 3])


def test_select_prompt_chunks_special(pa):
    """Ties, marked pages, overflowing scores, zero and non-finite queries, ids outside the pool, the uniform
    layout, for runs of tokens."""
    b = R.Batch(3, [60] * 3, [1600, 1000, 700], 4, 2, 64, 16, "f32")
    env, scale = b.envelopes()
    same = np.broadcast_to(env[:1, :1], env.shape).copy()
    _check_select(pa, b, 1, 1, 9, env=(same, np.ones_like(scale)))
    marked = scale.copy()
    marked[np.random.default_rng(0).uniform(size=scale.shape) < 0.1] = np.inf
    _check_select(pa, b, 1, 1, 9, env=(env, marked), uniform=True)
    _check_select(pa, b, 0, 0, 30, env=(env, np.where(np.isnan(scale), scale, np.float32(3e38))))
    b.q[0] = 0
    b.q[61, 1, 5] = np.nan
    b.q[122, 3, 0] = np.inf
    _check_select(pa, b, 0, 1, 9)
    b.table[0, 3], b.table[1, 20], b.table[0, 30] = b.P, -1, W.SENTINEL_MAX
    want = R.select(b.q64(), env, scale, b.table, b.rows(), 2, 16, 1, 2, 8)
    np.testing.assert_array_equal(_run_select(pa, b, env, scale, 1, 2, 8), want)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE


def _long_runs(seed, q_lens, pages, Hq, Hkv, D, dtype, q_pad=2):
    """Runs of tokens behind long prefixes over a small pool (many equal scores): at least 2^23 (token, query
    head, page) scores, which is where the tcgen05 kernel takes them."""
    assert sum(q_lens) * Hq * pages >= 1 << 23
    rng = np.random.default_rng(seed)
    b = R.Batch(seed, q_lens, q_lens, Hq, Hkv, D, 16, dtype, q_pad=q_pad)
    short = rng.integers(0, 3, len(q_lens))
    b.seq_lens = np.asarray([pages * 16 - int(x) * 37 - int(rng.integers(0, 16)) for x in short], np.int32)
    b.width, b.P = pages, 600
    b.table = rng.integers(0, b.P, (len(q_lens), pages)).astype(np.int32)
    hi = rng.integers(-127, 128, (b.P, Hkv, D)).astype(np.int8)
    lo = np.minimum(hi, rng.integers(-127, 128, (b.P, Hkv, D))).astype(np.int8)
    return b, (np.stack([lo, hi], 2), rng.uniform(0.5, 1, (b.P, Hkv)).astype(np.float32))


@pytest.mark.parametrize("q_lens,pages,Hq,Hkv,D,dtype", [
    ([2000, 1, 900, 700], 600, 4, 1, 128, "bf16"), ([500, 0, 460, 1], 1100, 8, 2, 64, "f16"),
    ([130, 1, 130], 2100, 16, 1, 128, "f32"), ([2000, 1, 1150], 900, 3, 1, 64, "bf16"),
    ([290], 1500, 20, 1, 128, "f16"), ([3300], 1300, 2, 2, 64, "bf16"), ([380], 700, 32, 1, 64, "bf16"),
    ([90, 15, 16, 2], 4300, 16, 2, 64, "bf16"), ([1000, 30], 600, 14, 2, 128, "bf16")])
def test_select_long_runs(pa, q_lens, pages, Hq, Hkv, D, dtype):
    b, env = _long_runs(pages, q_lens, pages, Hq, Hkv, D, dtype)
    _check_select(pa, b, 1, 2, 40, env=env)
    _check_select(pa, b, 0, 0, 3, env=env)


def test_select_long_runs_special(pa):
    """Ties, marked pages, overflowing scores, zero and non-finite queries, no scored page, non-causal, the
    uniform layout, ids outside the pool."""
    b, (env, scale) = _long_runs(1, [700, 700], 800, 8, 2, 64, "f32", q_pad=0)
    b.q[0] = 0
    b.q[61, 1, 5] = np.nan
    b.q[722, 3, 0] = np.inf
    _check_select(pa, b, 0, 1, 9, env=(env, scale))
    _check_select(pa, b, 3, 6, 9, env=(env, scale))
    _check_select(pa, b, 1, 1, 9, env=(env, scale), causal=False)
    _check_select(pa, b, 1, 1, 9, env=(env, scale), uniform=True)
    _check_select(pa, b, 1, 1, 9, env=(env, scale), q_offset=[-300, 90])
    same = np.broadcast_to(env[:1, :1], env.shape).copy()
    _check_select(pa, b, 1, 1, 9, env=(same, np.ones_like(scale)))
    marked = scale.copy()
    marked[np.random.default_rng(0).uniform(size=scale.shape) < 0.1] = np.inf
    _check_select(pa, b, 1, 1, 9, env=(env, marked))
    _check_select(pa, b, 0, 0, 30, env=(env, np.full_like(scale, 3e38)))
    b.table[0, 3], b.table[1, 20], b.table[0, 130] = b.P, -1, W.SENTINEL_MAX
    want = R.select(b.q64(), env, scale, b.table, b.rows(), 2, 16, 1, 2, 8)
    np.testing.assert_array_equal(_run_select(pa, b, env, scale, 1, 2, 8)[:b.T], want)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE


@pytest.mark.parametrize("D", [64, 128])
def test_select_long_runs_largest_scores(pa, D):
    """The largest scores, that differ by one, for a run of tokens."""
    b, (env, _) = _long_runs(D, [1400], 800, 8, 2, D, "bf16")
    rng = np.random.default_rng(D)
    sign = rng.choice([-1, 1], D)
    b.q[:] = W.bf16_bits_rne(np.broadcast_to(3.0 * sign, b.q.shape).astype(np.float32))
    env[:] = np.where(sign > 0, 127, -127).astype(np.int8)
    env[b.P // 2:] *= -1
    for p in range(b.P):
        d = rng.integers(0, D)
        env[p, :, :, d] -= np.sign(env[p, :, :, d]) * np.int8(rng.integers(0, 3))
    _check_select(pa, b, 1, 1, 30, env=(env, np.ones((b.P, b.Hkv), np.float32)))


@pytest.mark.parametrize("D", [64, 128])
def test_select_prompt_chunks_largest_scores(pa, D):
    """The largest scores, that differ by one, for a run of tokens."""
    b = R.Batch(D, [64], [200 * 16], 8, 2, D, 16, "bf16")
    rng = np.random.default_rng(D)
    sign = rng.choice([-1, 1], D)
    b.q[:] = W.bf16_bits_rne(np.broadcast_to(3.0 * sign, b.q.shape).astype(np.float32))
    env = np.broadcast_to(np.where(sign > 0, 127, -127).astype(np.int8), (b.P, b.Hkv, 2, D)).copy()
    env[b.P // 2:] *= -1
    for p in range(b.P):
        d = rng.integers(0, D)
        env[p, :, :, d] -= np.sign(env[p, :, :, d]) * np.int8(rng.integers(0, 3))
    _check_select(pa, b, 1, 1, 30, env=(env, np.ones((b.P, b.Hkv), np.float32)))


@pytest.mark.parametrize("pages,Hq", [(700, 8), (1500, 4), (3000, 16), (8000, 4)])
def test_select_prompt_chunks_long(pa, pages, Hq):
    """Runs of tokens behind long prefixes, many equal scores among them."""
    rng = np.random.default_rng(pages)
    b = R.Batch(pages, [70], [70], Hq, 2, 64, 16, "bf16")
    b.seq_lens = np.array([pages * 16 - 3], np.int32)
    b.width, b.P = pages, 2000
    b.table = rng.integers(0, b.P, (1, pages)).astype(np.int32)
    hi = rng.integers(-127, 128, (b.P, 2, 64)).astype(np.int8)
    lo = np.minimum(hi, rng.integers(-127, 128, (b.P, 2, 64))).astype(np.int8)
    _check_select(pa, b, 1, 2, 50, env=(np.stack([lo, hi], 2), rng.uniform(0.5, 1, (b.P, 2)).astype(np.float32)))


@pytest.mark.parametrize("B,pages,K,ps", [(2, 4097, 64, 16), (1, 20000, 128, 16), (3, 1025, 100, 64),
                                          (1, 49151, 700, 16), (5, 2047, 2000, 32)])
def test_select_long(pa, B, pages, K, ps):
    """Long sequences: envelopes drawn directly (many equal scores among them)."""
    rng = np.random.default_rng(pages)
    b = R.Batch(pages, [1] * B, [1] * B, 4, 1, 64, ps, "bf16")
    lens = pages * ps - rng.integers(0, ps, B) - ps * rng.integers(0, pages // 3, B)
    lens[0] = pages * ps
    b.seq_lens = lens.astype(np.int32)
    b.width, b.P = pages, 5000
    b.table = rng.integers(0, b.P, (B, pages)).astype(np.int32)
    hi = rng.integers(-127, 128, (b.P, 1, 64)).astype(np.int8)
    lo = np.minimum(hi, rng.integers(-127, 128, (b.P, 1, 64))).astype(np.int8)
    _check_select(pa, b, 1, 2, K, env=(np.stack([lo, hi], 2), rng.uniform(0.5, 1, (b.P, 1)).astype(np.float32)))


@pytest.mark.parametrize("Hkv,ps", [(1, 16), (3, 64), (8, 32)])
def test_select_rows_shorter_than_the_list(pa, Hkv, ps):
    """Tables no wider than top_k: every reachable page, for few tokens and for many; rows of no sequence stay."""
    for q_lens, seq_lens in (([1], [1]), ([3, 0, 1, 70], [200, 5, 90, 130]), ([600] * 9 + [1], [640, 600] * 5)):
        b = R.Batch(50, q_lens, seq_lens, 2 * Hkv, Hkv, 64, ps, "bf16", q_pad=5)
        W_ = b.width
        for K in (W_, W_ + 1, W_ + 37, 200):
            _check_select(pa, b, 0, 1, K)
        _check_select(pa, b, 0, 0, W_, causal=False)
        qo = [int(L) - 2 * n - 9 for n, L in zip(q_lens, b.seq_lens)]  # the first tokens see nothing
        _check_select(pa, b, 1, 0, W_, q_offset=qo)
    b = R.Batch(51, [4] * 3, [60, 4, 33], 2 * Hkv, Hkv, 64, ps, "f32")
    _check_select(pa, b, 0, 0, b.width, uniform=True)
    b = R.Batch(52, [1, 40], [300, 290], 2, 1, 64, 16, "bf16")
    b.table = np.ascontiguousarray(b.table[:, :3])
    b.width = 3
    env = b.envelopes()
    want = R.select(b.q64(), *env, b.table, b.rows(), 1, 16, 0, 0, 4)
    np.testing.assert_array_equal(_run_select(pa, b, *env, 0, 0, 4), want)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_SEQ_CLIPPED


def test_select_bad_pages(pa):
    """Ids outside the pool score 0 and are reported."""
    b = R.Batch(8, [2, 1], [800, 600], 4, 2, 128, 16, "bf16")
    env = b.envelopes()
    b.table[0, 3], b.table[1, 20], b.table[0, 30] = b.P, -1, W.SENTINEL_MAX
    want = R.select(b.q64(), *env, b.table, b.rows(), 2, 16, 1, 2, 8)
    np.testing.assert_array_equal(_run_select(pa, b, *env, 1, 2, 8), want)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE


# ----------------------------------------------------------------------------- attention over listed pages
def _lists(b, K, seed=0, causal=True, q_offset=None):
    """Random lists: distinct reachable pages in any order, some rows short, one empty."""
    rng = np.random.default_rng(seed)
    sel = np.full((b.T, b.Hkv, K), -1, np.int32)
    for t, (_, reach) in enumerate(b.rows(causal, q_offset)):
        np_ = -(-reach // b.ps)
        for h in range(b.Hkv):
            n = min(np_, K if rng.uniform() < 0.7 else rng.integers(0, K + 1))
            sel[t, h, :n] = rng.permutation(np_)[:n]
    return sel


def _run_attend(pa, b, sel, causal=True, q_offset=None, uniform=False, q=None, scale=None, stream=None):
    import torch
    d = b.device()
    q = d["q"] if q is None else q
    qo = None if q_offset is None else _t(q_offset, np.int32)
    full = np.full((q.shape[0], b.Hkv, sel.shape[-1]), 0, np.int32)
    full[:b.T] = sel
    out = torch.full(tuple(q.shape), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(tuple(q.shape[:-1]), 7.0, device="cuda")
    scale = b.D ** -0.5 if scale is None else scale
    if uniform:
        B = len(b.q_lens)
        u = lambda t: t.view(B, -1, *t.shape[1:])  # noqa: E731
        pa.paged_attn_fwd_sparse(u(q), d["k"], d["v"], d["table"], d["lens"], causal, qo, u(_t(full)), scale, u(out),
                                 u(lse))
    else:
        pa.paged_attn_fwd_sparse(q, d["k"], d["v"], d["table"], d["lens"], causal, qo, _t(full), scale, out, lse,
                                 q_start=d["q_start"])
    torch.cuda.synchronize()
    assert (out[b.T:] == 7.0).all() and (lse[b.T:] == 7.0).all()  # rows of no sequence are left as they were
    return _gpu.to_f64(out[:b.T], b.dtype), _gpu.to_f64(lse[:b.T], "f32")


def _check_attend(pa, b, sel, causal=True, q_offset=None, scale=None, **kw):
    out, lse = _run_attend(pa, b, sel, causal, q_offset, scale=scale, **kw)
    k, v = R.elems_to_f64(b.k, b.dtype), R.elems_to_f64(b.v, b.dtype)
    want = R.attend(b.q64(), k, v, b.table, b.rows(causal, q_offset), sel, b.ps, b.D ** -0.5 if scale is None else scale)
    _gpu.assert_close(out, want[0], b.dtype, "out")
    _gpu.assert_close(lse, want[1], b.dtype, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 16), (3, 3, 64, 32), (14, 2, 128, 64), (24, 1, 64, 16),
                                         (33, 1, 128, 32), (6, 2, 256, 16), (16, 1, 256, 64), (2, 2, 256, 32),
                                         (4, 4, 128, 16), (16, 1, 64, 64)])
def test_attend(pa, dtype, Hq, Hkv, D, ps):
    b = R.Batch(Hq * D, [1, 3, 0, 1, 5], [1, 12 * ps, 9, 7 * ps + 5, 9 * ps + 1], Hq, Hkv, D, ps, dtype, q_pad=2)
    for K in (1, 7, 12):
        _check_attend(pa, b, _lists(b, K))


def test_attend_few_rows_long_lists(pa):
    """One token over hundreds of pages (the split over the list), in each type."""
    for dtype, D in (("bf16", 128), ("f16", 64), ("f32", 128), ("bf16", 256)):
        for n in (1, 2):
            b = R.Batch(D, [1] * n, [6000, 4000][:n], 8, 2, D, 16, dtype)
            _check_attend(pa, b, _lists(b, 300))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(7, 1, 64), (8, 2, 128), (3, 1, 256)])
def test_attend_few_rows_split_lists(pa, dtype, Hq, Hkv, D):
    """Lists split over clusters of every size, parts of them empty or cut short, entries repeated."""
    b = R.Batch(D + 1, [1, 0, 2], [5000, 90, 700], Hq, Hkv, D, 16, dtype, q_pad=1)
    for K in (15, 16, 33, 65, 129, 300):
        sel = _lists(b, K, seed=K)
        sel[1, 0, :K // 2] = -1
        sel[2, 0, -3:] = sel[2, 0, 0]
        _check_attend(pa, b, sel)
    assert pa.paged_attn_last_error_word() == 0


# Runs of tokens long enough, with the lists below, for the kernel that reads the union of their lists.
CHUNKS = [1, 230, 0, 16, 15, 1, 129]
CHUNK_LENS = [90, 500, 5, 16, 700, 64, 129]


def _shares(pa, b, K, uniform=False, scale=0.1):
    import torch
    code = {"bf16": pa.PA_BF16, "f16": pa.PA_F16, "f32": pa.PA_F32}[b.dtype]
    B = len(b.q_lens)
    return pa.paged_attn_sparse_shares_pages(B, b.T // B if uniform else b.T, b.Hq, b.Hkv, b.D, b.ps, b.width, K, scale,
                                             torch.cuda.get_device_properties(0).multi_processor_count, code,
                                             not uniform)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 16), (4, 4, 64, 32), (14, 2, 64, 64), (16, 1, 128, 16),
                                         (3, 1, 128, 64), (10, 2, 128, 32), (18, 1, 64, 16), (8, 1, 128, 32),
                                         (16, 2, 128, 64), (4, 1, 128, 64), (64, 1, 128, 16), (2, 2, 64, 16)])
def test_attend_prompt_chunks(pa, dtype, Hq, Hkv, D, ps):
    """Runs of tokens whose lists are read together, beside short sequences in the same call."""
    b = R.Batch(Hq * D + ps, CHUNKS, CHUNK_LENS, Hq, Hkv, D, ps, dtype, q_pad=3)
    assert _shares(pa, b, 40)
    for K in (1, 5, 40):
        _check_attend(pa, b, _lists(b, K))
    qo = [max(0, L - n - 7) for n, L in zip(CHUNKS, CHUNK_LENS)]
    qo[1] = -6  # a chunk whose first tokens see nothing
    _check_attend(pa, b, _lists(b, 40, q_offset=qo), q_offset=qo)
    _check_attend(pa, b, _lists(b, 40, causal=False), causal=False)


def test_attend_prompt_chunks_uniform(pa):
    for n in (15, 16, 50, 64):
        b = R.Batch(n, [n] * 8, [n, 200, 130, 180, 199, 64, 65, 66], 8, 2, 128, 16, "bf16")
        assert _shares(pa, b, 13, True) == (n >= 16) and not _shares(pa, b, 13, True, -0.2)
        _check_attend(pa, b, _lists(b, 13), uniform=True)
        _check_attend(pa, b, _lists(b, 13), uniform=True, scale=-0.2)
        _check_attend(pa, b, _lists(b, 13), uniform=True, scale=3.0)  # the row maximum moves far


def test_attend_prompt_chunks_any_list(pa):
    """Repeated entries count again, in one tile of a chunk or in all; ids outside the pool read as zeros."""
    for dtype in ("bf16", "f16"):
        b = R.Batch(31, CHUNKS, CHUNK_LENS, 8, 2, 128, 16, dtype)
        assert _shares(pa, b, 40)
        sel = _lists(b, 40)
        sel[40, 1, :4] = [2, 0, 2, 2]
        sel[45, 0] = -7
        sel[45, 0, :9] = [-1, W.SENTINEL_MAX, -2**31, 1, 1, 99, 1, 0, -7]
        sel[300, 0] = -1
        _check_attend(pa, b, sel)
        assert pa.paged_attn_last_error_word() == 0
        sel[:, :, 1] = sel[:, :, 0]
        _check_attend(pa, b, sel)
        b.table[1, 2], b.table[4, 7] = b.P, -1
        sel = _lists(b, 40, seed=3)
        sel[:, :, 1:][sel[:, :, 1:] == 2] = -1
        sel[:, :, 0] = 2
        _check_attend(pa, b, sel)
        assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE


def test_attend_prompt_chunks_non_finite(pa):
    """An infinity or a NaN in a key or a value reaches the rows that list its page and see its key, and
    no other row of the tile."""
    for dtype, inf, nan in (("bf16", 0x7F80, 0x7FC0), ("f16", 0x7C00, 0x7E00)):
        b = R.Batch(32, [64] * 8, [200] * 8, 8, 2, 128, 16, dtype)
        assert _shares(pa, b, 13, True)
        sel = np.zeros((512, 2, 13), np.int32) - 1
        sel[:, :, :3] = [1, 4, 8]
        sel[20:23, :, 1] = 6
        sel[30, 1, 1] = 5
        clean = _run_attend(pa, b, sel, uniform=True)[0]
        b.v[b.table[0, 6], 2, 0, 3] = nan
        b.k[b.table[0, 5], 7, 1, 9] = nan
        b.v[b.table[0, 9], 10, 1, 64] = inf  # position 154: no token of head 1 lists page 9
        b.v[b.table[0, 8], 15, 0, 11] = inf  # position 143
        sel[5, 0, :3] = [1, 4, 9]            # token 5 sees positions up to 141: no key of page 9
        out = _run_attend(pa, b, sel, uniform=True)[0]
        bad = ~np.isfinite(out)
        want = np.zeros_like(bad)
        want[20:23, :4, 3] = True             # page 6, kv head 0, one column
        want[30, 4:, :] = True                # a NaN score: every column
        want[7:64, :4, 11] = True             # tokens that see position 143 (136 + 7)
        np.testing.assert_array_equal(bad, want)
        same = ~want.any(-1)
        same[5, :4] = False
        _gpu.assert_close(out[same], clean[same], dtype, "rows without them")


def test_attend_masks(pa):
    """Non-causal, explicit offsets (one puts every key out of reach), the uniform layout, a view of q,
    a negative and a zero scale."""
    import torch
    for dtype in ("bf16", "f32"):
        b = R.Batch(2, [4, 4, 4], [190, 30, 150], 8, 2, 128, 16, dtype)
        _check_attend(pa, b, _lists(b, 6, causal=False), causal=False)
        qo = [60, -9, 146]
        _check_attend(pa, b, _lists(b, 6, q_offset=qo), q_offset=qo)
        sel = _lists(b, 6)
        _check_attend(pa, b, sel, uniform=True)
        _check_attend(pa, b, sel, scale=-0.1)
        _check_attend(pa, b, sel, scale=0.0)
        fused = torch.full((b.T, 12, 128), float("nan"), dtype=b.device()["q"].dtype, device="cuda")
        fused[:, 2:10] = b.device()["q"]
        _check_attend(pa, b, sel, q=fused[:, 2:10])


def test_attend_any_list(pa):
    """Entries out of reach and negative ones list nothing, repeated ones count again; an empty list gives
    0 and -inf."""
    for dtype in ("f16", "f32"):
        b = R.Batch(9, [2, 1], [150, 80], 4, 2, 128, 16, dtype)
        sel = _lists(b, 9)
        sel[0, 0] = [-1, 3, W.SENTINEL_MAX, 3, 9, -2**31, 0, 10, 3]
        sel[1, 1] = -1
        sel[2, 0] = 99
        _check_attend(pa, b, sel)
    assert pa.paged_attn_last_error_word() == 0


def test_attend_bad_pages(pa):
    """A listed page whose id is outside the pool reads as zeros and is reported."""
    for dtype in ("bf16", "f32"):
        b = R.Batch(8, [2, 1], [300, 200], 4, 2, 128, 16, dtype)
        b.table[0, 3], b.table[1, 2] = b.P, -1
        sel = _lists(b, 8)
        sel[:, :, 0], sel[:, :, 1] = 3, 2
        _check_attend(pa, b, sel)
        assert pa.paged_attn_last_error_word() == pa.ERRBIT_PAGE_RANGE


def test_attend_every_page_is_dense_attention(pa):
    """Listing every page gives what the dense call gives, to its bars."""
    import torch
    b = R.Batch(12, [1] * 4, [300, 17, 64, 1], 16, 4, 128, 16, "bf16")
    d = b.device()
    K = b.width
    sel = torch.arange(K, dtype=torch.int32, device="cuda").repeat(4, 1, 4, 1).contiguous()
    q = d["q"].view(4, 1, 16, 128)
    out, lse = torch.empty_like(q), torch.empty(4, 1, 16, device="cuda")
    pa.paged_attn_fwd_sparse(q, d["k"], d["v"], d["table"], d["lens"], True, None, sel, 128 ** -0.5, out, lse)
    dense, dl = pa.attention(q, d["k"], d["v"], d["table"], d["lens"], causal=True, want_lse=True)
    _gpu.assert_close(_gpu.to_f64(out, "bf16"), _gpu.to_f64(dense, "bf16"), "bf16", "out")
    _gpu.assert_close(_gpu.to_f64(lse, "f32"), _gpu.to_f64(dl, "f32"), "bf16", "lse")


def test_attend_nan_reaches_its_rows_only(pa):
    """A NaN in a listed page gives NaN in the rows that list it, and only there."""
    b = R.Batch(13, [1, 1], [200, 200], 4, 2, 128, 16, "bf16")
    sel = np.zeros((2, 2, 3), np.int32)
    sel[:] = [1, 4, 12]
    b.k[b.table[0, 4], 2, 1, 3] = 0x7FC0
    out, lse = _run_attend(pa, b, sel)
    bad = np.isnan(out).all(-1)
    assert bad[0, 2:].all() and not np.isnan(out[0, :2]).any() and not np.isnan(out[1]).any()


# ----------------------------------------------------------------------------- the step as it is used
def _serve(pa, dtype, Hq, Hkv, D, ps, plan, top_k, graph=False, stream=None):
    """Run a serving loop: ``plan`` is a list of new-token counts per request and step.  Every step's
    output is checked against the plain implementation on the host's own copy of the state."""
    import torch
    rng = np.random.default_rng(17)
    B, steps = len(plan[0]), len(plan)
    total_len = np.asarray(plan).sum(0)
    width = int(-(-total_len.max() // ps)) + 1
    P = int((-(-total_len // ps)).sum()) + 5
    T = int(np.asarray(plan).sum(1).max()) + 3
    pool = (P, ps, Hkv, D)
    nan = {"f32": np.float32(np.nan), "f16": np.uint16(0x7E00), "bf16": np.uint16(0x7FC0)}[dtype]
    zero = np.zeros(pool, np.float32 if dtype == "f32" else np.uint16)
    hk, hv = zero + nan, zero + nan
    k, v = W.host_to_torch(hk, dtype).cuda(), W.host_to_torch(hv, dtype).cuda()
    env, scale = pa.page_envelopes(k)
    henv, hscale = np.zeros((P, Hkv, 2, D), np.int8), np.zeros((P, Hkv), np.float32)
    i32 = lambda a: _t(np.asarray(a), np.int32)  # noqa: E731
    free = rng.permutation(P).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    lens = np.zeros(B, np.int32)
    count = P
    d_free, d_count, d_table, d_lens = i32(free), i32([count]), _t(table), i32(lens)
    d_new, d_qo, d_qs, d_slots = i32([0] * B), i32([0] * B), i32([0] * (B + 1)), i32([0] * T)
    tdt = W.torch_dtype(dtype)
    qkv = torch.zeros((T, Hq + 2 * Hkv, D), dtype=tdt, device="cuda")
    sel = torch.zeros((T, Hkv, top_k), dtype=torch.int32, device="cuda")
    out, lse = torch.zeros((T, Hq, D), dtype=tdt, device="cuda"), torch.zeros((T, Hq), device="cuda")

    def step():
        pa.paged_attn_step_tables(d_lens, d_new, d_free, d_count, d_table, d_lens, d_qo, d_qs, d_slots, d_count, ps, P)
        pa.paged_attn_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], d_slots, k, v, env, scale)
        pa.paged_attn_select_pages(qkv[:, :Hq], env, scale, d_table, d_lens, True, d_qo, 1, 1, sel, ps, q_start=d_qs)
        pa.paged_attn_fwd_sparse(qkv[:, :Hq], k, v, d_table, d_lens, True, d_qo, sel, D ** -0.5, out, lse,
                                 q_start=d_qs)

    run = step
    if graph:
        d_new.zero_()
        step()  # first calls outside the capture; an idle step changes nothing
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    for n, new in enumerate(plan):
        new = np.asarray(new, np.int32)
        h = R.random_elems(rng, (T, Hq + 2 * Hkv, D), dtype)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        d_new.copy_(_t(new))
        qkv.copy_(W.host_to_torch(h, dtype))
        torch.cuda.synchronize()
        if stream is None:
            run()
        else:
            with torch.cuda.stream(stream):
                run()
        torch.cuda.synchronize()
        want = R.step_tables(lens, new, free, count, table, T, ps, P)
        assert not want["refused"]
        np.testing.assert_array_equal(d_slots.cpu().numpy(), want["slots"])
        np.testing.assert_array_equal(d_table.cpu().numpy(), want["table"])
        table, lens, count = want["table"], want["seq_lens"], int(want["free_left"][0])
        R.append(h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:], want["slots"], hk, hv, dtype, henv, hscale)
        np.testing.assert_array_equal(env.cpu().numpy(), henv)
        np.testing.assert_array_equal(scale.cpu().numpy(), hscale)
        rows = R.token_rows(new.tolist(), lens, width, ps, True, None)
        m = int(new.sum())
        q64 = R.elems_to_f64(h[:m, :Hq], dtype)
        ref_sel = R.select(q64, henv, hscale, table, rows, Hkv, ps, 1, 1, top_k)
        np.testing.assert_array_equal(sel.cpu().numpy()[:m], ref_sel)
        ref = R.attend(q64, R.elems_to_f64(hk, dtype), R.elems_to_f64(hv, dtype), table, rows, ref_sel, ps, D ** -0.5)
        _gpu.assert_close(_gpu.to_f64(out, dtype)[:m], ref[0], dtype, f"step {n} out")
        _gpu.assert_close(_gpu.to_f64(lse, "f32")[:m], ref[1], dtype, f"step {n} lse")
    assert pa.paged_attn_last_error_word() == 0


PLAN = [[130, 0, 7, 64], [1, 90, 1, 1], [1, 1, 0, 1], [3, 1, 1, 1], [1, 1, 33, 1]]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", [("bf16", 8, 2, 128, 16), ("f16", 3, 3, 64, 32), ("f32", 4, 1, 256, 16),
                                               ("bf16", 14, 2, 256, 32)])
def test_serving_loop(pa, dtype, Hq, Hkv, D, ps):
    _serve(pa, dtype, Hq, Hkv, D, ps, PLAN, top_k=4)


def test_serving_loop_as_a_graph(pa):
    """The four calls captured once; every replay takes the state the last one left."""
    _serve(pa, "bf16", 8, 2, 128, 16, PLAN, top_k=4, graph=True)


def test_serving_loop_on_another_stream(pa):
    import torch
    _serve(pa, "bf16", 8, 2, 128, 16, PLAN, top_k=4, stream=torch.cuda.Stream())


def test_attention_sparse(pa):
    """The convenience call: selection and attention, with its allocations on a stream of its own."""
    import torch
    b = R.Batch(21, [1, 1], [700, 400], 8, 2, 128, 16, "bf16")
    env = b.envelopes()
    d = b.device()
    e, s = _t(env[0]), _t(env[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, lse, sel = pa.attention_sparse(d["q"], d["k"], d["v"], e, s, d["table"], d["lens"], top_k=12,
                                        q_start=d["q_start"], want_lse=True, want_pages=True, stream=st)
    torch.cuda.synchronize()
    ref_sel = R.select(b.q64(), *env, b.table, b.rows(), 2, 16, 1, 2, 12)
    np.testing.assert_array_equal(sel.cpu().numpy(), ref_sel)
    k, v = R.elems_to_f64(b.k, "bf16"), R.elems_to_f64(b.v, "bf16")
    ref = R.attend(b.q64(), k, v, b.table, b.rows(), ref_sel, 16, 128 ** -0.5)
    _gpu.assert_close(_gpu.to_f64(out, "bf16"), ref[0], "bf16", "out")
    _gpu.assert_close(_gpu.to_f64(lse, "f32"), ref[1], "bf16", "lse")


def test_same_bits_on_every_run(pa):
    b = R.Batch(22, [1, 2, 1], [5000, 900, 3000], 8, 2, 128, 16, "bf16")
    sel = _lists(b, 100)
    first = _run_attend(pa, b, sel)
    for _ in range(3):
        again = _run_attend(pa, b, sel)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_malformed_q_start(pa):
    """A sequence whose q_start entries are out of range is skipped and reported."""
    import torch
    b = R.Batch(23, [1, 1, 1], [300, 200, 100], 4, 2, 64, 16, "bf16")
    d = b.device()
    env = b.envelopes()
    for qs in ([0, 1, 2, 9], [0, 1, -5, 3], [0, 9, 2, 3]):
        sel = torch.full((3, 2, 4), -9, dtype=torch.int32, device="cuda")
        q_start = _t(qs, np.int32)
        pa.paged_attn_select_pages(d["q"], _t(env[0]), _t(env[1]), d["table"], d["lens"], True, None, 1, 1, sel, 16,
                                   q_start=q_start)
        good = sel.clamp(min=-1)
        out = torch.empty_like(d["q"])
        pa.paged_attn_fwd_sparse(d["q"], d["k"], d["v"], d["table"], d["lens"], True, None, good, 0.1, out, None,
                                 q_start=q_start)
        assert pa.paged_attn_last_error_word() & ~pa.ERRBIT_QSTART == 0


def test_pools_past_2_31_bytes(pa):
    """The whole step over the last pages of pools of 4.7 GB: byte and element offsets pass 31 bits."""
    import torch
    Hq, Hkv, D, ps, P = 8, 8, 128, 16, 144000
    b = R.Batch(41, [40, 1], [300, 200], Hq, Hkv, D, ps, "bf16", spare=0)
    low = P - b.P
    k = torch.zeros((P, ps, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert low * ps * Hkv * D > 1 << 31
    env, scale = pa.page_envelopes(k)
    table = np.where(b.table < b.P, b.table + low, b.table).astype(np.int32)
    # every token through append, the first ones as an earlier call
    k_host, v_host = b.k.copy(), b.v.copy()
    nan = np.isnan(R.elems_to_f64(k_host, "bf16"))
    k_host[nan], v_host[nan] = 0, 0
    d = {n: _t(x) for n, x in (("table", table), ("lens", b.seq_lens), ("q_start", b.q_start))}
    for part in (0, 1):
        slots, rows = [], []
        for s, n in enumerate(b.q_lens):
            L = int(b.seq_lens[s])
            for x in (range(L - n) if part == 0 else range(L - n, L)):
                slots.append(int(table[s, x // ps]) * ps + x % ps)
                rows.append((int(b.table[s, x // ps]), x % ps))
        pick = tuple(np.array(rows).T)
        pa.paged_attn_append(W.host_to_torch(k_host[pick], "bf16").cuda(), W.host_to_torch(v_host[pick], "bf16").cuda(),
                             _t(slots, np.int32), k, v, env, scale)
    want_env, want_scale = b.envelopes()
    live = b.live.any(-1)
    np.testing.assert_array_equal(env[low:].cpu().numpy()[live], want_env[live])
    np.testing.assert_array_equal(scale[low:].cpu().numpy()[live], want_scale[live])
    assert not env[:low].any() and not k[:low].any()
    q = W.host_to_torch(b.q, "bf16").cuda()
    out, lse, sel = pa.attention_sparse(q, k, v, env, scale, d["table"], d["lens"], top_k=6, q_start=d["q_start"],
                                        want_lse=True, want_pages=True)
    want = R.select(b.q64(), want_env, want_scale, b.table, b.rows(), Hkv, ps, 1, 2, 6)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)
    ref = R.attend(b.q64(), R.elems_to_f64(b.k, "bf16"), R.elems_to_f64(b.v, "bf16"), b.table, b.rows(), want, ps,
                   D ** -0.5)
    _gpu.assert_close(_gpu.to_f64(out, "bf16"), ref[0], "bf16", "out")
    _gpu.assert_close(_gpu.to_f64(lse, "f32"), ref[1], "bf16", "lse")


@pytest.mark.parametrize("n", [1, 200])
def test_sequences_longer_than_their_table(pa, n):
    """seq_lens past the table row are clipped to it and reported, for single tokens and for runs."""
    b = R.Batch(42, [n] * 3, [300, 260, 290], 8, 2, 128, 16, "bf16")
    env = b.envelopes()
    full = b.table
    b.width = 16
    b.table = np.ascontiguousarray(full[:, :16])
    sel = _lists(b, 12)
    _check_attend(pa, b, sel)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_SEQ_CLIPPED
    want = R.select(b.q64(), *env, b.table, b.rows(), 2, 16, 1, 2, 6)
    np.testing.assert_array_equal(_run_select(pa, b, *env, 1, 2, 6)[:b.T], want)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_SEQ_CLIPPED


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qs", [[0, 40, 20, 80], [0, 10, 70, 60], [0, 81, 81, 81], [-1, 80, 80, 80], [0, 0, 90, 80]])
def test_every_malformed_range_is_reported(pa, dtype, qs):
    """Rows that a malformed sequence shares with a sound one do not hide it, whichever kernel runs."""
    import torch
    K = 8 if dtype == "f32" else 60
    b = R.Batch(46, [1] * 3, [1600, 1200, 1500], 8, 2, 128, 16, dtype, q_pad=77)
    d = b.device()
    env, scale = (_t(x) for x in b.envelopes())
    q_start = _t(qs, np.int32)
    sel = torch.full((80, 2, K), -1, dtype=torch.int32, device="cuda")
    pa.paged_attn_select_pages(d["q"], env, scale, d["table"], d["lens"], True, None, 1, 1, sel, 16, q_start=q_start)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_QSTART
    out = torch.empty_like(d["q"])
    pa.paged_attn_fwd_sparse(d["q"], d["k"], d["v"], d["table"], d["lens"], True, None, sel, 0.1, out, None,
                             q_start=q_start)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_QSTART


def test_malformed_ranges_among_long_runs(pa):
    """The same where the long runs' kernels take the first launch: sound sequences keep their results."""
    import torch
    b = R.Batch(47, [700, 3, 697], [1600, 1200, 1500], 64, 2, 128, 16, "bf16")
    assert b.T * 64 * b.width >= 1 << 23 and _shares(pa, b, 60)
    env, scale = b.envelopes()
    args = [_t(x) for x in (env, scale, b.table, b.seq_lens)]
    q = b.device()["q"]
    sel = torch.full((b.T, 2, 60), -9, dtype=torch.int32, device="cuda")
    q_start = _t([0, 700, 699, b.T], np.int32)
    pa.paged_attn_select_pages(q, *args, True, None, 1, 1, sel, 16, q_start=q_start)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_QSTART
    want = R.select(b.q64()[:40], env, scale, b.table, b.rows()[:40], 2, 16, 1, 1, 60)
    np.testing.assert_array_equal(sel[:40].cpu().numpy(), want)
    d = b.device()
    pa.paged_attn_fwd_sparse(q, d["k"], d["v"], d["table"], d["lens"], True, None, sel, 0.1, torch.empty_like(q), None,
                             q_start=q_start)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_QSTART


def test_more_sequences_than_threads(pa):
    """One token among 6000 sequences of none, the last of them malformed."""
    import torch
    B = 6000
    d = dict(dtype=torch.int32, device="cuda")
    q_start = torch.zeros(B + 1, **d)
    q_start[17:] = 1
    lens, table = torch.full((B,), 40, **d), torch.arange(3, **d).repeat(B, 1)
    k = torch.randn((3, 16, 1, 64), device="cuda")
    env, scale = torch.zeros((3, 1, 2, 64), dtype=torch.int8, device="cuda"), torch.zeros((3, 1), device="cuda")
    q, sel, out = torch.randn((1, 1, 64), device="cuda"), torch.empty((1, 1, 3), **d), torch.empty((1, 1, 64), device="cuda")
    for bad in (False, True):
        if bad:
            q_start[B] = 2
        for call in (lambda: pa.paged_attn_select_pages(q, env, scale, table, lens, True, None, 1, 1, sel, 16, q_start=q_start),
                     lambda: pa.paged_attn_fwd_sparse(q, k, k, table, lens, True, None, sel, 0.1, out, None, q_start=q_start)):
            call()
            assert pa.paged_attn_last_error_word() == (pa.ERRBIT_QSTART if bad else 0)
        assert sel.flatten().tolist() == [0, 1, 2] and out.isfinite().all()


@pytest.mark.parametrize("n", [1, 300])
def test_select_nan_scale(pa, n):
    """A page whose scale is a NaN has no bound: it comes first, as one with +inf does."""
    b = R.Batch(44, [n] * 2, [6000, 5000], 8, 2, 128, 16, "bf16")
    env, scale = b.envelopes()
    marked = scale.copy()
    for s, j in ((0, 7), (0, 100), (1, 50), (1, 200)):
        marked[b.table[s, j]] = np.inf
        scale[b.table[s, j]] = np.nan
    want = R.select(b.q64(), env, marked, b.table, b.rows(), 2, 16, 1, 2, 9)
    np.testing.assert_array_equal(_run_select(pa, b, env, scale, 1, 2, 9)[:b.T], want)
    assert pa.paged_attn_last_error_word() == 0


@pytest.mark.parametrize("D,G,n,pages", [(256, 24, 1, 500), (256, 40, 2, 1500), (256, 24, 1, 49152), (128, 17, 1, 49152),
                                         (256, 4, 70, 900)])
def test_select_wide_groups(pa, D, G, n, pages):
    """Many heads of head_dim 256, up to the longest row."""
    rng = np.random.default_rng(D + G + pages)
    b = R.Batch(45, [n], [n], G, 1, D, 16, "bf16")
    b.seq_lens = np.array([pages * 16 - 5], np.int32)
    b.width, b.P = pages, 3000
    b.table = rng.integers(0, b.P, (1, pages)).astype(np.int32)
    hi = rng.integers(-127, 128, (b.P, 1, D)).astype(np.int8)
    lo = np.minimum(hi, rng.integers(-127, 128, (b.P, 1, D))).astype(np.int8)
    _check_select(pa, b, 1, 2, 60, env=(np.stack([lo, hi], 2), rng.uniform(0.5, 1, (b.P, 1)).astype(np.float32)))


def test_two_streams_at_once(pa):
    """Calls on two streams share nothing: each gives what it gives alone."""
    import torch
    b = R.Batch(43, [1, 60, 1], [3000, 900, 700], 8, 2, 128, 16, "bf16")
    d = b.device()
    env, scale = (_t(x) for x in b.envelopes())
    sets = []
    for i in range(2):
        q = W.host_to_torch(R.random_elems(np.random.default_rng(i), b.q.shape, "bf16"), "bf16").cuda()
        sets.append([q, torch.empty(b.T, 2, 20, dtype=torch.int32, device="cuda"), torch.empty_like(q)])

    def call(q, sel, out):
        pa.paged_attn_select_pages(q, env, scale, d["table"], d["lens"], True, None, 1, 2, sel, 16, q_start=d["q_start"])
        pa.paged_attn_fwd_sparse(q, d["k"], d["v"], d["table"], d["lens"], True, None, sel, 0.1, out, None,
                                 q_start=d["q_start"])
    alone = []
    for s in sets:
        call(*s)
        torch.cuda.synchronize()
        alone.append((s[1].clone(), s[2].clone()))
    streams = [torch.cuda.Stream() for _ in sets]
    for s in sets:
        s[1].zero_()
        s[2].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                call(*s)
    torch.cuda.synchronize()
    for s, (sel, out) in zip(sets, alone):
        assert torch.equal(s[1], sel) and torch.equal(s[2], out)


@pytest.mark.parametrize("graph", [False, True])
def test_what_follows_follows_both_launches(pa, graph):
    """Where a call is two launches side by side, the next work on the stream sees all its rows and may
    overwrite them."""
    import torch
    b = R.Batch(48, [700, 3, 1, 697], [1600, 1200, 900, 1500], 64, 2, 128, 16, "bf16")
    assert b.T * 64 * b.width >= 1 << 23 and _shares(pa, b, 40)
    env, scale = (_t(x) for x in b.envelopes())
    d = b.device()
    sel = torch.full((b.T, 2, 40), -9, dtype=torch.int32, device="cuda")
    out, lists, outs = torch.empty_like(d["q"]), [], []

    def step():
        pa.paged_attn_select_pages(d["q"], env, scale, d["table"], d["lens"], True, None, 1, 2, sel, 16,
                                   q_start=d["q_start"])
        lists.append(sel.clone())
        pa.paged_attn_fwd_sparse(d["q"], d["k"], d["v"], d["table"], d["lens"], True, None, lists[-1], 0.1, out, None,
                                 q_start=d["q_start"])
        outs.append(out.clone())
        sel.fill_(-9)
        out.fill_(7)
    step()
    torch.cuda.synchronize()
    want = R.select(b.q64(), env.cpu().numpy(), scale.cpu().numpy(), b.table, b.rows(), 2, 16, 1, 2, 40)
    np.testing.assert_array_equal(lists[0].cpu().numpy(), want)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                step()
        for _ in range(3):
            g.replay()
    else:
        for _ in range(30):
            step()
    torch.cuda.synchronize()
    for x, y in zip(lists, outs):
        assert torch.equal(x, lists[0]) and torch.equal(y, outs[0])
    assert (sel == -9).all() and (out == 7).all()
    assert pa.paged_attn_last_error_word() == 0
