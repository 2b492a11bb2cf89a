"""Plain implementations of the calls over selected pages (numpy, 64 bits), written from the header's
definitions, and seeded inputs for their tests."""
from __future__ import annotations

import numpy as np

from paged_kv_cache_201_gb300 import workloads as W

NP_F = {"f32": np.float32, "f16": np.float16}


def elems_to_f64(a, dtype):
    """Host elements (float32, or uint16 bits of f16 / bf16) as float64 (exact)."""
    if dtype == "f32":
        return a.astype(np.float64)
    if dtype == "f16":
        return a.view(np.float16).astype(np.float64)
    return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def random_elems(rng, shape, dtype):
    return W._normal_elems(rng, int(np.prod(shape)), dtype).reshape(shape)


# ----------------------------------------------------------------------------- tables
def step_tables(cached, new, free_pages, free_count, table, total, ps, num_pages):
    """The step's outputs, request after request.  Returns a dict; ``table`` is not changed."""
    table = table.copy()
    width = table.shape[1]
    count = min(max(free_count, 0), len(free_pages))
    refused, bad_page = count != free_count, False
    pages_asked = tokens_asked = taken = 0
    lens, starts, slots = [], [0], []
    for b, (c, n) in enumerate(zip(cached.tolist(), new.tolist())):
        usable = c >= 0 and n >= 0 and -(-(c + n) // ps) <= width
        served = False
        if usable:
            have, want = -(-c // ps), -(-(c + n) // ps)
            pages_asked += want - have
            tokens_asked += n
            served = (want == have or pages_asked <= count) and tokens_asked <= total
        if served:
            for p in range(have, want):
                table[b, p] = free_pages[count - 1 - taken]
                taken += 1
            for x in range(c, c + n):
                page = int(table[b, x // ps])
                ok = 0 <= page < num_pages
                bad_page |= not ok
                slots.append(page * ps + x % ps if ok else -1)
        elif n != 0 or c < 0:
            refused = True
        lens.append(c + n if served else c)
        starts.append(len(slots))
    slots += [-1] * (total - len(slots))
    i32 = lambda v: np.asarray(v, np.int32)  # noqa: E731
    return {"table": table, "seq_lens": i32(lens), "q_offset": cached.astype(np.int32), "q_start": i32(starts),
            "slots": i32(slots), "free_left": i32([count - taken]), "refused": refused, "bad_page": bad_page}


# ----------------------------------------------------------------------------- append
def envelope(keys):
    """(int8 [2, D], float32 scale) of keys [rows, D] (float64 holding exact elements)."""
    if not np.isfinite(keys).all():
        return np.zeros((2, keys.shape[1]), np.int8), np.float32(np.inf)
    lo, hi = keys.min(0).astype(np.float32), keys.max(0).astype(np.float32)
    a = np.float32(max(np.abs(lo).max(), np.abs(hi).max()))
    if a == 0:
        return np.zeros((2, keys.shape[1]), np.int8), np.float32(0)
    q = np.rint((np.stack([lo, hi]) / a) * np.float32(127))
    return q.astype(np.int8), np.float32(a / np.float32(127))


def append(k_new, v_new, slots, k, v, dtype, env=None, scale=None):
    """In place on host element arrays k, v [P, ps, Hkv, D] (and env, scale)."""
    P, ps, Hkv, D = k.shape
    end = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < P * ps:
            k[s // ps, s % ps], v[s // ps, s % ps] = k_new[t], v_new[t]
            end[s // ps] = max(end.get(s // ps, 0), s % ps)
    if env is not None:
        for page, r in end.items():
            rows = elems_to_f64(k[page, :r + 1], dtype)
            for h in range(Hkv):
                env[page, h], scale[page, h] = envelope(rows[:, h])


# ----------------------------------------------------------------------------- queries and their reach
def token_rows(q_lens, seq_lens, width, ps, causal, q_offset):
    """[(sequence, reach)] of the packed query tokens."""
    rows = []
    for b, n in enumerate(q_lens):
        L = min(max(int(seq_lens[b]), 0), width * ps)
        off = int(q_offset[b]) if q_offset is not None else L - n
        for i in range(n):
            rows.append((b, min(L, max(0, off + i + 1)) if causal else L))
    return rows


# ----------------------------------------------------------------------------- selection
def select(q, env, scale, table, rows, Hkv, ps, sink, local, K):
    """sel [T, Hkv, K] for q [T, Hq, D] (float64 holding exact elements)."""
    T, Hq, D = q.shape
    G = Hq // Hkv
    P = env.shape[0]
    sel = np.full((T, Hkv, K), -1, np.int32)
    for t, (b, reach) in enumerate(rows):
        np_ = -(-reach // ps)
        for h in range(Hkv):
            if np_ <= K:
                sel[t, h, :np_] = np.arange(np_)
                continue
            x = q[t, h * G:(h + 1) * G].astype(np.float32)
            a = np.abs(x).max()
            qi = np.zeros(x.shape, np.int64)
            if np.isfinite(x).all() and a > 0:
                qi = np.rint((x / a) * np.float32(127)).astype(np.int64)
            pages = table[b, :np_]
            ok = (pages >= 0) & (pages < P)
            e = np.where(ok[:, None, None], env[np.where(ok, pages, 0), h].astype(np.int64), 0)
            s = (np.maximum(qi, 0) @ e[:, 1].T + np.minimum(qi, 0) @ e[:, 0].T).max(0)
            sc = np.where(ok, scale[np.where(ok, pages, 0), h], np.float32(0))
            with np.errstate(invalid="ignore"):
                score = np.where(np.isinf(sc), np.float32(np.inf), s.astype(np.float32) * sc)
            mid = np.arange(sink, np_ - local)
            order = mid[np.argsort(-score[mid].astype(np.float64), kind="stable")]
            got = sorted([*range(sink), *order[:K - sink - local], *range(np_ - local, np_)])
            sel[t, h] = got
    return sel


# ----------------------------------------------------------------------------- attention
def attend(q, k, v, table, rows, sel, ps, scale):
    """(out [T, Hq, D], lse [T, Hq]) for float64 q and pools; an out-of-range page reads as zeros."""
    T, Hq, D = q.shape
    P, _, Hkv, _ = k.shape
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    for t, (b, reach) in enumerate(rows):
        for h in range(Hkv):
            kk, vv = [], []
            for j in sel[t, h].tolist():
                if j < 0 or j * ps >= reach:
                    continue
                n = min(ps, reach - j * ps)
                page = int(table[b, j])
                if 0 <= page < P:
                    kk.append(k[page, :n, h])
                    vv.append(v[page, :n, h])
                else:
                    kk.append(np.zeros((n, D)))
                    vv.append(np.zeros((n, D)))
            if not kk:
                continue
            kk, vv = np.concatenate(kk), np.concatenate(vv)
            s = q[t, h * G:(h + 1) * G] @ kk.T * scale
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            out[t, h * G:(h + 1) * G] = (w @ vv) / w.sum(-1, keepdims=True)
            lse[t, h * G:(h + 1) * G] = (m + np.log(w.sum(-1, keepdims=True)))[:, 0]
    return out, lse


# ----------------------------------------------------------------------------- inputs
class Batch:
    """A ragged batch over shuffled pages.  Rows past a sequence's end, pages of nobody and block-table
    slots past a sequence's pages hold garbage (NaN elements, unmapped ids)."""

    def __init__(self, seed, q_lens, seq_lens, Hq, Hkv, D, ps, dtype, spare=3, q_pad=0):
        rng = np.random.default_rng(seed)
        self.q_lens, self.seq_lens = list(q_lens), np.asarray(seq_lens, np.int32)
        self.Hq, self.Hkv, self.D, self.ps, self.dtype = Hq, Hkv, D, ps, dtype
        B = len(q_lens)
        need = -(-np.maximum(self.seq_lens, 0) // ps)
        self.width = int(max(1, need.max() + 1)) if B else 1
        self.P = int(need.sum()) + spare
        ids = rng.permutation(self.P).astype(np.int32)
        self.table = np.full((B, self.width), W.SENTINEL_MAX, np.int32)
        self.table[np.arange(self.width)[None] < need[:, None]] = ids[:int(need.sum())]
        shape = (self.P, ps, Hkv, D)
        nan = {"f32": np.float32(np.nan), "f16": np.uint16(0x7E00), "bf16": np.uint16(0x7FC0)}[dtype]
        self.k, self.v = random_elems(rng, shape, dtype), random_elems(rng, shape, dtype)
        live = np.zeros((self.P, ps), bool)
        for b in range(B):
            for j in range(int(need[b])):
                live[self.table[b, j], :int(self.seq_lens[b]) - j * ps] = True
        self.k[~live] = nan
        self.v[~live] = nan
        self.live = live
        self.T = int(sum(q_lens))
        self.q = random_elems(rng, (self.T + q_pad, Hq, D), dtype)
        self.q_start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)

    def envelopes(self):
        """env, scale of every page over its live rows (pages of nobody: garbage)."""
        env = np.full((self.P, self.Hkv, 2, self.D), 99, np.int8)
        scale = np.full((self.P, self.Hkv), np.nan, np.float32)
        kf = elems_to_f64(self.k, self.dtype)
        for p in range(self.P):
            n = int(self.live[p].sum())
            for h in range(self.Hkv):
                if n:
                    env[p, h], scale[p, h] = envelope(kf[p, :n, h])
        return env, scale

    def rows(self, causal=True, q_offset=None):
        return token_rows(self.q_lens, self.seq_lens, self.width, self.ps, causal, q_offset)

    def q64(self):
        return elems_to_f64(self.q, self.dtype)[:self.T]

    def device(self):
        import torch
        g = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        e = lambda a: W.host_to_torch(a, self.dtype).cuda()  # noqa: E731
        return {"q": e(self.q), "k": e(self.k), "v": e(self.v), "table": g(self.table), "lens": g(self.seq_lens),
                "q_start": g(self.q_start)}
