"""Plain implementations of the 4-bit cache and of the calls that share, free and move pages: 64-bit
floats and Python lists, from the definitions in include/paged_attn.h."""
import numpy as np

SCALES = np.array([c * 2.0 ** -17 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 18) for c in range(0xDF)])


def quantise(x):
    """Codes u (0 .. 15) and scale bytes of rows x [..., D] (float64)."""
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
    g = x.reshape(*x.shape[:-1], -1, 16)
    t = np.minimum(np.abs(g).max(-1) / 7, SCALES[-1])
    i = np.clip(np.searchsorted(SCALES, t, side="right") - 1, 0, len(SCALES) - 2)
    down, up = t - SCALES[i], SCALES[i + 1] - t
    c = np.where((up < down) | ((up == down) & (i % 2 == 1)), i + 1, i)
    s = SCALES[c][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(s > 0, 8 + np.clip(np.rint(g / s), -7, 7), 8)
    return u.reshape(x.shape).astype(np.uint8), c.astype(np.uint8)


def cut(pool, ps, D):
    """Views of a pool [..., 9 ps D / 8]: K codes, V codes [..., ps, D / 2], K scales, V scales [..., ps, D / 16]."""
    h, f = ps * D // 2, ps * D // 16
    parts = (pool[..., :h], pool[..., h:2 * h], pool[..., 2 * h:2 * h + f], pool[..., 2 * h + f:])
    return [p.reshape(*p.shape[:-1], ps, -1) for p in parts]


def write(pool, slots, k, v, ps):
    """Rows k, v [T, Hkv, D] into the slots of a pool [P, Hkv, 9 ps D / 8], in place."""
    D = k.shape[-1]
    h, f = ps * D // 2, ps * D // 16
    for side, x in enumerate((k, v)):
        u, c = quantise(x)
        packed = u[..., 0::2] | (u[..., 1::2] << 4)
        for t, s in enumerate(slots):
            if 0 <= s < pool.shape[0] * ps:
                p, r = divmod(int(s), ps)
                a, b = side * h + r * (D // 2), 2 * h + side * f + r * (D // 16)
                pool[p, :, a:a + D // 2] = packed[t]
                pool[p, :, b:b + D // 16] = c[t]


def values(pool, ps, D):
    """K and V [P, Hkv, ps, D] of a pool, float64."""
    kc, vc, ks, vs = cut(pool, ps, D)
    out = []
    for codes, sc in ((kc, ks), (vc, vs)):
        u = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D).astype(np.float64) - 8
        out.append(u * np.repeat(SCALES[np.minimum(sc, 0xDE)], 16, -1))
    return out


def attention(q, pool, ps, table, lens, starts, causal, q_offset, scale):
    """Rows of packed q [T, Hq, D]: out, lse, how far float32 sums may be off in the score (nats) and in the
    output, and the weighted mean of |v| (float64); rows of no sequence hold NaN."""
    T, Hq, D = q.shape
    P, Hkv, _ = pool.shape
    k, v = values(pool, ps, D)
    G = Hq // Hkv
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    off, room, mass = np.zeros((T, Hq)), np.zeros((T, Hq, 1)), np.zeros((T, Hq, D))
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        L = min(max(int(lens[b]), 0), table.shape[1] * ps)
        ids = table[b, :-(-L // ps)]
        good = (ids >= 0) & (ids < P)
        kk, vv = (np.where(good[:, None, None, None], x[np.where(good, ids, 0)], 0.0).transpose(1, 0, 2, 3)
                  .reshape(Hkv, -1, D)[:, :L] for x in (k, v))
        first = int(q_offset[b]) if q_offset is not None else L - n
        for i in range(n):
            t = starts[b] + i
            r = min(max(first + i + 1, 0), L) if causal else L
            if r == 0:
                out[t], lse[t] = 0.0, -np.inf
                continue
            for h in range(Hq):
                s = kk[h // G, :r] @ q[t, h] * scale
                top = s.max()
                w = np.exp(s - top)
                out[t, h] = w @ vv[h // G, :r] / w.sum()
                mass[t, h] = w @ np.abs(vv[h // G, :r]) / w.sum()
                lse[t, h] = top + np.log(w.sum())
                # products summed in float32 over D terms (a truncating adder: 2^-23 each), the factor's and the
                # exponential's roundings on the score
                off[t, h] = (np.abs(kk[h // G, :r]) @ np.abs(q[t, h])).max() * abs(scale) * D * 2.0 ** -23 + \
                    np.abs(s).max() * 2.0 ** -22 + 2.0 ** -20
                room[t, h] = 2 * off[t, h] * np.abs(vv[h // G, :r]).max()
    return out, lse, off, room, mass


# ----------------------------------------------------------------------------- pages
def pages_of(length, W, ps):
    return -(-min(max(length, 0), W * ps) // ps)


def fork(parents, children, prefix, table, lens, shares, free, count, ps, P):
    """Sequentially, on lists and arrays of its own; also whether something was refused or out of the pool."""
    table, lens, shares = table.copy(), list(lens), list(shares)
    B, W = table.shape
    old, F = list(lens), min(max(count, 0), len(free))
    refused, bad = F != count, False
    copies, named, need, taken = [], set(), 0, 0
    for i, (a, c) in enumerate(zip(parents, children)):
        copies.append([-1, -1])
        if a == -1:
            continue
        ok = 0 <= a < B and 0 <= c < B and a != c and old[c] == 0 and c not in named
        if 0 <= c < B:
            named.add(c)
        ok = ok and (prefix is None or prefix[i] >= 0)
        if not ok:
            refused = True
            continue
        n = min(max(old[a], 0), W * ps)
        if prefix is not None:
            n = min(n, prefix[i])
        need += n % ps != 0
        if n % ps and need > F:
            refused = True
            continue
        for j in range(n // ps):
            p = table[c, j] = table[a, j]
            if 0 <= p < P:
                shares[p] += 1
            else:
                bad = True
        if n % ps:
            to = free[F - 1 - taken]
            taken += 1
            table[c, n // ps] = to
            if 0 <= table[a, n // ps] < P and 0 <= to < P:
                copies[-1] = [table[a, n // ps], to]
            else:
                bad = True
        lens[c] = n
    return dict(table=table, lens=lens, shares=shares, copies=copies, left=F - taken, refused=refused, bad=bad)


def free(rows, table, lens, shares, stack, count, ps, P):
    lens, shares, stack = list(lens), list(shares), list(stack)
    B, W = table.shape
    F, cap = min(max(count, 0), len(stack)), len(stack)
    refused, bad = F != count, False
    asked = []
    for r in rows:
        if r == -1 or r in asked:
            continue
        if not 0 <= r < B:
            refused = True
            continue
        asked.append(r)
    for r in reversed(asked):
        for j in reversed(range(pages_of(lens[r], W, ps))):
            p = table[r, j]
            if not 0 <= p < P:
                bad = True
            elif shares[p] > 0:
                shares[p] -= 1
            else:
                if F < cap:
                    stack[F] = p
                    F += 1
                else:
                    refused = True
        lens[r] = 0
    return dict(lens=lens, shares=shares, stack=stack, left=F, refused=refused, bad=bad)


def compact(table, lens, shares, stack, count, ps, P):
    table, shares, stack = table.copy(), list(shares), list(stack)
    B, W = table.shape
    F = min(max(count, 0), len(stack))
    refused = F != count
    listed = [(b, j) for b in range(B) for j in range(pages_of(lens[b], W, ps))]
    used = sorted({int(table[b, j]) for b, j in listed if 0 <= table[b, j] < P})
    bad = any(not 0 <= table[b, j] < P for b, j in listed) or any(not 0 <= p < P for p in stack[:F])
    idle = [p for p in stack[:F] if 0 <= p < P]
    refused |= len(set(idle)) != len(idle) or bool(set(idle) & set(used))
    idle = sorted(set(idle) - set(used))
    k = 0
    while k < min(len(used), len(idle)) and idle[k] < used[-1 - k]:
        k += 1
    moves = list(zip(used[len(used) - k:], idle[:k]))
    where = list(range(P))
    for a, b in moves:
        where[a] = b
        shares[b], shares[a] = shares[a], 0
    for b, j in listed:
        if 0 <= table[b, j] < P:
            table[b, j] = where[table[b, j]]
    now = sorted(idle[k:] + [a for a, _ in moves], reverse=True)
    stack[:len(now)] = now
    return dict(table=table, shares=shares, stack=stack, left=len(now), moves=moves, page_map=where, refused=refused,
                bad=bad)
