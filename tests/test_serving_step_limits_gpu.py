"""Calls over selected pages that the documentation allows and that sit at its edges: slots named twice, empty
batches, sound sequences beside malformed ones, the kernels for runs of tokens on two streams and again and again."""
import numpy as np
import pytest

from paged_kv_cache_201_gb300 import workloads as W
from tests import _gpu
from tests import _sparse_ref as R
from tests.test_serving_step_gpu import (_append_case, _check_attend, _check_select, _lists, _raw, _run_append,  # noqa: F401
                                         _run_attend, _shares, _t, pa)

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


# ----------------------------------------------------------------------------- malformed query ranges
def _claims(qs, T):
    """Sound sequences that claim each row."""
    claims = [[] for _ in range(T)]
    for b, (a, e) in enumerate(zip(qs, qs[1:])):
        if 0 <= a <= e <= T:
            for t in range(a, e):
                claims[t].append(b)
    return claims


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,qs,found", [
    (3, [0, 1, 2, 9], {0, 1}), (3, [0, 1, -5, 3], {0}), (3, [0, 9, 2, 3], {2}), (80, [0, 10, 70, 60], set(range(70))),
    (80, [0, 20, 90, 80], set(range(20))), (80, [-1, 80, 80, 80], set()), (80, [0, 40, 20, 80], set(range(20))),
    (80, [0, 0, 500, 4], set()), (80, [0, 500, 40, 80], set())])
def test_rows_beside_malformed_ranges(pa, dtype, T, qs, found):  # noqa: F811
    """A malformed sequence's rows stay as they were.  Another sequence's rows are its own or stay, too (`found`:
    those that are certainly there, ahead of the first malformed entry); a row that two claim is either's."""
    import torch
    b = R.Batch(T, [1] * 3, [1600, 1200, 1500], 8, 2, 128, 16, dtype, q_pad=T - 3)
    q64, (env, scale), K = R.elems_to_f64(b.q, dtype), b.envelopes(), 9
    k, v = R.elems_to_f64(b.k, dtype), R.elems_to_f64(b.v, dtype)
    d = b.device()
    q_start = _t(qs, np.int32)
    sel = torch.full((T, 2, K), -9, dtype=torch.int32, device="cuda")
    pa.paged_attn_select_pages(d["q"], _t(env), _t(scale), d["table"], d["lens"], True, None, 1, 1, sel, 16,
                               q_start=q_start)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_QSTART
    lists = np.broadcast_to(np.arange(K, dtype=np.int32), (T, 2, K)).copy()
    out, lse = torch.full_like(d["q"], 7.0), torch.full((T, 8), 7.0, device="cuda")
    pa.paged_attn_fwd_sparse(d["q"], d["k"], d["v"], d["table"], d["lens"], True, None, _t(lists), 0.1, out, lse,
                             q_start=q_start)
    assert pa.paged_attn_last_error_word() == pa.ERRBIT_QSTART
    sel, out, lse = sel.cpu().numpy(), _gpu.to_f64(out, dtype), _gpu.to_f64(lse, "f32")
    for t, claim in enumerate(_claims(qs, T)):
        if t in found or not (sel[t] == -9).all():
            wants = []
            for s in claim:
                n = qs[s + 1] - qs[s]
                row = [(s, min(int(b.seq_lens[s]), int(b.seq_lens[s]) - n + t - qs[s] + 1))]
                wants.append(R.select(q64[t:t + 1], env, scale, b.table, row, 2, 16, 1, 1, K)[0])
            assert any(np.array_equal(sel[t], w) for w in wants), (t, claim)
        if t not in found and (out[t] == 7.0).all() and (lse[t] == 7.0).all():
            continue
        assert claim
        fits = []
        for s in claim:
            n = qs[s + 1] - qs[s]
            row = [(s, int(b.seq_lens[s]) - n + t - qs[s] + 1)]
            want = R.attend(q64[t:t + 1], k, v, b.table, row, lists[t:t + 1], 16, 0.1)
            atol, rtol = _gpu.TOL[dtype]
            fits.append((np.abs(out[t] - want[0][0]) <= atol + rtol * np.abs(want[0][0])).all()
                        and (np.abs(lse[t] - want[1][0]) <= atol + rtol * np.abs(want[1][0])).all())
        assert any(fits), (t, claim)


# ----------------------------------------------------------------------------- the kernels for runs of tokens
def _two_launches(dtype="bf16", seed=48):
    """A batch that both of a call's launches work on, in selection (2^23 scores) and attention."""
    return R.Batch(seed, [700, 3, 1, 697], [1600, 1200, 900, 1500], 64, 2, 128, 16, dtype)


def test_runs_of_tokens_on_two_streams_at_once(pa):  # noqa: F811
    """Each call gives what it gives alone, its tensor memory and its second launch its own."""
    import torch
    b = _two_launches()
    assert b.T * 64 * b.width >= 1 << 23 and _shares(pa, b, 40)
    d = b.device()
    env, scale = (_t(x) for x in b.envelopes())
    sets = []
    for i in range(2):
        q = W.host_to_torch(R.random_elems(np.random.default_rng(i), b.q.shape, "bf16"), "bf16").cuda()
        sets.append([q, torch.empty(b.T, 2, 40, dtype=torch.int32, device="cuda"), torch.empty_like(q)])

    def call(q, sel, out):
        pa.paged_attn_select_pages(q, env, scale, d["table"], d["lens"], True, None, 1, 2, sel, 16, q_start=d["q_start"])
        pa.paged_attn_fwd_sparse(q, d["k"], d["v"], d["table"], d["lens"], True, None, sel, 0.1, out, None,
                                 q_start=d["q_start"])
    alone = []
    for s in sets:
        call(*s)
        torch.cuda.synchronize()
        alone.append((s[1].clone(), s[2].clone()))
        s[1].zero_()
        s[2].zero_()
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                call(*s)
    torch.cuda.synchronize()
    for s, (sel, out) in zip(sets, alone):
        assert torch.equal(s[1], sel) and torch.equal(s[2], out)
    assert pa.paged_attn_last_error_word() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_runs_of_tokens_give_the_same_bits_on_every_run(pa, dtype):  # noqa: F811
    import torch
    b = _two_launches(dtype, 49)
    assert _shares(pa, b, 40)
    d, sel = b.device(), _t(_lists(b, 40))
    first = None
    for _ in range(4):
        out, lse = torch.full_like(d["q"], 7.0), torch.full((b.T, 64), 7.0, device="cuda")
        pa.paged_attn_fwd_sparse(d["q"], d["k"], d["v"], d["table"], d["lens"], True, None, sel, 0.1, out, lse,
                                 q_start=d["q_start"])
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


# ----------------------------------------------------------------------------- tables and batches of a serving loop
@pytest.mark.parametrize("columns", [300, 1100, 5000])
@pytest.mark.parametrize("q_lens,seq_lens", [
    ([1] * 9, [500, 3, 900, 64, 1, 700, 17, 333, 1200]),       # single tokens, lengths spread widely
    ([260, 1, 1, 40], [900, 500, 7, 300]),                     # chunks beside single tokens
    ([90] + [1] * 130, [400] + [37 + 11 * i for i in range(130)])])  # single tokens outnumber a chunk's
def test_tables_wider_than_their_sequences(pa, q_lens, seq_lens, columns):  # noqa: F811
    """A loop's table is as wide as its longest request may become: the columns past a sequence's pages are not read."""
    b = R.Batch(columns, q_lens, seq_lens, 8, 2, 128, 16, "f16", q_pad=2)
    b.table = np.concatenate([b.table, np.full((len(q_lens), columns), W.SENTINEL_MAX, np.int32)], 1)
    b.width += columns
    for K in (7, 20):
        _check_select(pa, b, 1, 2, K)
        _check_attend(pa, b, _lists(b, K))
    assert pa.paged_attn_last_error_word() == 0


@pytest.mark.parametrize("q_lens", [[1, 1], [300, 300]])
@pytest.mark.parametrize("exponent", [5, 15, 23, 25, 27])
@pytest.mark.parametrize("dtype,D", [("f16", 128), ("f16", 64), ("bf16", 128)])
def test_largest_scores(pa, q_lens, exponent, dtype, D):  # noqa: F811
    """Scores up to 2^27, the largest shared by every fifth key, a smaller one met before it: the output is the mean
    of those keys' values.  The weights are then equal (the others below 2^-22 of them), so the bar is the rounding of the output and of
    float32 sums: half a step and 2 n 2^-24 of the largest value."""
    n = 600
    b = R.Batch(D, q_lens, [n] * 2, 8, 2, D, 16, dtype)
    el = (lambda x: x.astype(np.float16).view(np.uint16)) if dtype == "f16" else \
        (lambda x: W.bf16_bits_rne(x.astype(np.float32).ravel()).reshape(x.shape))
    key = np.zeros(b.k.shape)
    peak = np.zeros(n, bool)
    peak[100::5] = True
    for s in range(2):
        at = np.arange(n)
        key[b.table[s, at // 16], at % 16, :, 0] = np.where(peak, 1.0, np.where(at == 3, 0.5, 0.0))[:, None] * 2.0 ** 12
    b.k[:] = el(key)
    q = np.zeros(b.q.shape)
    q[..., 0] = 2.0 ** (exponent - 12)
    b.q[:] = el(q)
    b.v[~b.live] = 0
    K = -(-n // 16)
    sel = np.broadcast_to(np.arange(K, dtype=np.int32), (b.T, 2, K)).copy()
    if q_lens[0] > 1:
        assert _shares(pa, b, K, scale=1.0)
    out, lse = _run_attend(pa, b, sel, causal=False, scale=1.0)
    v = R.elems_to_f64(b.v, dtype)
    eps = 2.0 ** (-11 if dtype == "f16" else -8)
    for s in range(2):
        at = np.flatnonzero(peak)
        want = v[b.table[s, at // 16], at % 16].mean(0)  # [Hkv, D]
        rows = slice(int(b.q_start[s]), int(b.q_start[s + 1]))
        got = out[rows].reshape(-1, 2, 4, D)
        err = np.abs(got - want[None, :, None])
        assert (err <= eps * np.abs(want[None, :, None]) + 2 * n * 2.0 ** -24 * np.abs(v).max()).all(), err.max()
        top = 2.0 ** exponent + np.log(peak.sum())
        assert np.abs(lse[rows] - top).max() <= 2.0 ** -21 * top
    assert pa.paged_attn_last_error_word() == 0
