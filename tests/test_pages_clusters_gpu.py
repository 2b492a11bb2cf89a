"""Frees by clusters of CTAs where CTAs start late or go through several rounds, against sequential lists
(tests/_kv4_ref.py).  Everything is a whole number and must match exactly."""
import numpy as np
import pytest

from tests import _kv4_ref as R
from tests.test_pages_gpu import _full, _state, _t, pa  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,width", [(60, 40), (300, 40), (900, 90)])
def test_free_beside_other_work(pa, B, width):
    """Four to sixteen CTAs of a cluster, set up while the multiprocessors are taken, again and again."""
    import torch
    s = _state(B + width, B, width, 16, empty=0.05, shared=0.8)
    rows = s["rng"].permutation(B)
    want = R.free(list(rows), s["table"], s["lens"], s["shares"], s["stack"], s["count"], 16, s["P"])
    want = [_t(want[k]) for k in ("lens", "shares", "stack")] + [_t([want["left"]])]
    rows, table, lens, count = _t(rows), _t(s["table"]), _t(s["lens"]), _t([s["count"]])
    shares0, stack0 = _t(s["shares"]), _t(s["stack"])
    other, x = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda").bfloat16()
    torch.cuda.synchronize()
    wrong = _full(1, 0)
    for _ in range(100):
        with torch.cuda.stream(other):
            for _ in range(3):
                torch.mm(x, x)
        shares, stack = shares0.clone(), stack0.clone()
        lens_out, left = _full(B), _full(1)
        pa.paged_attn_free(rows, table, lens, lens_out, shares, stack, count, left, 16)
        for got, w in zip((lens_out, shares, stack, left), want):
            wrong += (got != w).any()
    assert int(wrong) == 0
    assert pa.paged_attn_last_error_word() == 0


def _rounds(seed, B, width, P, draw):
    """Rows of `width` full pages of 16, listed by draw(rng) -> [B, width]; a row more holds no tokens."""
    rng = np.random.default_rng(seed)
    table = draw(rng).astype(np.int32)
    shares = np.bincount(table.ravel(), minlength=P) - 1
    idle = rng.permutation(np.nonzero(shares < 0)[0])
    stack = np.full(P, -9, np.int32)
    stack[:len(idle)] = idle
    return dict(table=table, lens=np.full(B, width * 16, np.int32), shares=np.maximum(shares, 0).astype(np.int32), stack=stack,
                count=len(idle), ps=16, P=P, B=B, rng=rng)


def _check_free(pa, s, rows):
    want = R.free(list(rows), s["table"], s["lens"], s["shares"], s["stack"], s["count"], 16, s["P"])
    lens, shares, free = _t(s["lens"]), _t(s["shares"]), _t(s["stack"])
    lens_out, left = _full(s["B"]), _full(1)
    pa.paged_attn_free(_t(rows), _t(s["table"]), lens, lens_out, shares, free, _t([s["count"]]), left, 16)
    for got, w in ((lens_out, want["lens"]), (shares, want["shares"]), (free, want["stack"]), (left, [want["left"]])):
        np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(w, np.int32))
    assert not want["refused"] and not want["bad"] and pa.paged_attn_last_error_word() == 0


# A cluster takes 262144 listed pages a round, the last ones first.
@pytest.mark.parametrize("B,width", [(1100, 500), (600, 500), (70, 8000)])
def test_free_in_rounds(pa, B, width):
    """Two and three rounds: pages that nobody shares, pages of one round, and pages whose owners are in several."""
    listed = B * width
    P = listed + 1000

    def mixed(rng):
        t = rng.permutation(P)[:listed].reshape(B, width)
        for b in rng.permutation(B)[:B // 2]:  # a prompt in common with any row, early or late
            o, n = rng.integers(0, B), rng.integers(1, width)
            t[b, :n] = t[o, :n]
        return t
    s = _rounds(B, B, width, P, mixed)
    _check_free(pa, s, np.arange(B))
    _check_free(pa, s, s["rng"].permutation(B))
    _check_free(pa, s, s["rng"].permutation(B)[:B - 3])  # some owners stay


def test_free_in_rounds_some_without_sharing(pa):
    """Of three rounds the first, the second, the last or none has shared pages; and one page list for all rows."""
    B, width = 1200, 500
    P = B * width + 10
    for near in ((0, 100), (550, 650), (1100, 1200), None):
        def draw(rng):
            t = rng.permutation(P)[:B * width].reshape(B, width)
            if near:
                for b in range(near[0] + 1, near[1]):
                    t[b, :width // 2] = t[near[0], :width // 2]
            return t
        _check_free(pa, _rounds(3, B, width, P, draw), np.arange(B))
    s = _rounds(4, B, width, P, lambda rng: np.broadcast_to(rng.permutation(P)[:width], (B, width)).copy())
    _check_free(pa, s, np.arange(B))
