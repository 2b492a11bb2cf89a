"""Cases of the 4-bit cache and of the calls that share, free and move its pages.

A 4-bit pool holds, for every page and kv head, K and V codes of 4 bits and a scale of 8 bits for 16
elements (``paged_attn_append_kv4``); ``paged_attn_gather_kv4`` reads rows back as the values they stand
for and ``paged_attn_fwd_kv4`` attends over them.  ``paged_attn_fork`` lets a new sequence share another
one's pages, ``paged_attn_free`` gives a sequence's pages back, ``paged_attn_compact`` gathers the used
pages at the pool's start, and ``paged_attn_copy_pages`` moves the contents for the first and the last.

``own`` selects what ``run`` computes: the operators' plain form (elementary torch operations) or the
library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}
MAX_SCALE = 7168.0


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's rows of 256 sequences (8 kv heads of 128), a few rows of padding
        dict(name="rows_decode_256", op="rows", batch=256, chunk=1, pads=5, kv_heads=8, head_dim=128, page_size=16,
             length=512, dtype="bf16"),
        # prefill chunks of up to 2048 tokens in large pages, sliced out of a QKV projection
        dict(name="rows_chunk_8192", op="rows", batch=4, chunk=2048, pads=0, kv_heads=8, head_dim=128, page_size=64,
             length=8192, dtype="f16"),
        # a few tokens each of short sequences, three heads to a group: the smallest call
        dict(name="attend_odd_5", op="attend", batch=5, chunk=3, q_heads=6, kv_heads=2, head_dim=64, page_size=16,
             length=200, dtype="f16"),
        # decode of 256 ragged sequences of up to 4096 tokens
        dict(name="attend_decode_256", op="attend", batch=256, chunk=1, q_heads=32, kv_heads=8, head_dim=128,
             page_size=16, length=4096, dtype="bf16"),
        # one very long context, one new token: few rows, a long axis
        dict(name="attend_long_1", op="attend", batch=1, chunk=1, q_heads=32, kv_heads=8, head_dim=128, page_size=32,
             length=131072, dtype="bf16"),
        # prefill chunks of 512 tokens behind long prefixes
        dict(name="attend_chunk_1024", op="attend", batch=2, chunk=512, q_heads=32, kv_heads=8, head_dim=128,
             page_size=16, length=8192, dtype="bf16"),
        # four answers to one prompt: its pages shared, its last page copied, and given back later
        dict(name="fork_prompt_4", op="fork", parents=1, children=4, page_size=16, length=1000, layers=2, kv_heads=8,
             head_dim=128, pools="kv4"),
        # a beam-search step of 64 prompts with three more beams each
        dict(name="fork_beams_192", op="fork", parents=64, children=3, page_size=16, length=4096, layers=4, kv_heads=8,
             head_dim=128, pools="kv4"),
        # a few requests of a small server end
        dict(name="free_8", op="free", batch=32, rows=8, shared=0.25, page_size=16, length=2000),
        # a thousand of them at once, half with a prompt in common with others
        dict(name="free_1024", op="free", batch=1024, rows=1024, shared=0.5, page_size=16, length=4096),
        # a small pool's pages moved together
        dict(name="compact_2048", op="compact", pages=2048, batch=32, used=0.4, page_size=16, layers=2, kv_heads=8,
             head_dim=128, pools="kv4"),
        # a large pool, half empty after a burst of requests, in 16 bits
        dict(name="compact_32768", op="compact", pages=32768, batch=256, used=0.5, page_size=16, layers=1, kv_heads=8,
             head_dim=128, pools="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "rows", "attend", "attend", "attend", "fork", "free", "compact"])
    ps = rng.choice([16, 32, 64])
    head_dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "rows":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        batch = _log_int(rng, 1, 512)
        chunk = rng.choice([1, _log_int(rng, 2, 2048)])
        while batch * chunk * hkv * head_dim * ESIZE[dtype] > 8192 * 8 * 128 * 2:
            batch, chunk = max(1, batch // 2), max(1, (chunk * 2) // 3)
        length = max(chunk + 1, min(_log_int(rng, 64, 16384), (1 << 27) // (batch * hkv * head_dim)))
        return dict(op=op, batch=batch, chunk=chunk, pads=rng.choice([0, 0, rng.randint(1, 9)]), kv_heads=hkv,
                    head_dim=head_dim, page_size=ps, length=length, dtype=dtype)
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16, 24])
        batch = _log_int(rng, 1, 256)
        chunk = rng.choice([1, 1, _log_int(rng, 2, 512)])
        length = max(chunk, _log_int(rng, 17, 131072))

        def cost():
            return max(batch * length * hkv * head_dim / (256 * 4096 * 8 * 128),
                       batch * chunk * length * hkv * group * head_dim / (1024 * 8192 * 32 * 128))
        while cost() > 1:
            batch, chunk, length = max(1, batch * 2 // 3), max(1, chunk * 2 // 3), max(chunk, length * 3 // 4)
        return dict(op=op, batch=batch, chunk=chunk, q_heads=group * hkv, kv_heads=hkv, head_dim=head_dim,
                    page_size=ps, length=length, dtype=rng.choice(["bf16", "f16"]))
    pools = rng.choice(["kv4", "kv4", "bf16"])
    if op == "fork":
        parents, children = _log_int(rng, 1, 64), rng.randint(1, 6)
        length = _log_int(rng, 1, 4096)
        while parents * (children + 1) * (length / ps + 1) > 64 * 4 * 257:
            parents = max(1, parents * 2 // 3)
        layers = rng.randint(1, 4)
        while layers > 1 and parents * (length / ps + children + 1) * layers * _page_bytes(pools, ps, hkv, head_dim) > 1e9:
            layers -= 1
        return dict(op=op, parents=parents, children=children, page_size=ps, length=length, layers=layers, kv_heads=hkv,
                    head_dim=head_dim, pools=pools)
    if op == "free":
        batch = _log_int(rng, 1, 1024)
        return dict(op=op, batch=batch, rows=rng.randint((batch + 1) // 2, batch), shared=rng.choice([0.0, 0.25, 0.5]),
                    page_size=ps, length=_log_int(rng, 1, 256 * ps))
    pages, layers = _log_int(rng, 64, 32768), rng.randint(1, 2)
    while pages > 64 and pages * layers * _page_bytes(pools, ps, hkv, head_dim) > 32768 * 65536:
        pages = pages * 2 // 3
    return dict(op=op, pages=pages, batch=max(1, min(pages // 4, _log_int(rng, 1, 256))), used=rng.uniform(0.1, 0.9),
                page_size=ps, layers=layers, kv_heads=hkv, head_dim=head_dim, pools=pools)


# ----------------------------------------------------------------------------- inputs
def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _i32(n, fill=0):
    return torch.full(n if isinstance(n, tuple) else (n,), fill, dtype=torch.int32, device="cuda")


def _page_bytes(pools, ps, hkv, d):
    return ps * hkv * d * 9 // 8 if pools == "kv4" else 2 * ps * hkv * d * 2


def _page_tables(rng, lens, width, ps):
    """Block table [B, width] for sequences of these lengths over shuffled pages 1..; page 0 belongs to
    nobody, and slots past a sequence's pages hold -1.  Returns (table, pool pages)."""
    need = -(-lens // ps)
    total = int(need.sum())
    ids = rng.permutation(total).astype(np.int32) + 1
    table = np.full((len(lens), width), -1, np.int32)
    table[np.arange(width)[None] < need[:, None]] = ids
    return table, total + 1


def _batch(case, rng):
    """Lengths of a batch: new tokens a sequence (all of the chunk, or ragged), then all its tokens.  The
    case sets the lengths and the seed their order."""
    B, chunk = case["batch"], case["chunk"]
    spread = np.random.default_rng(B * chunk + case["length"])
    new = np.full(B, 1) if chunk == 1 else spread.integers((chunk + 1) // 2, chunk + 1, B)
    new[0] = chunk
    lens = np.maximum(new, (case["length"] * spread.uniform(0.4, 1.0, B)).astype(np.int64))
    lens[0] = case["length"]
    order = rng.permutation(B)
    return new[order].astype(np.int64), lens[order].astype(np.int64)


def _keys(gen, shape, dtype):
    """Key or value rows as a projection gives them: unit noise, and a few head-wide channels of larger
    size and shifted mean."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    d = torch.arange(shape[-1], device="cuda")
    return x.mul_(1 + 2 * (d % 37 == 5)).add_(1.5 * (d % 53 == 7)).to(dtype)


def _fill_kv4(gen, pool, ps, d):
    """A pool's blocks as appends leave them."""
    P, hkv, _ = pool.shape
    step = max(1, (1 << 25) // (hkv * ps * d))
    for part in pool.split(step):
        kc, vc, ks, vs = _parts(part, ps, d)
        for codes, scales in ((kc, ks), (vc, vs)):
            c, s = _quantise(_keys(gen, (part.shape[0], hkv, ps, d), torch.float32))
            codes.copy_(_packed(c))
            scales.copy_(_scale_byte(s))


def prepare(case, seed):
    rng = np.random.default_rng([seed, 73])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"rows": _prepare_rows, "attend": _prepare_attend, "fork": _prepare_fork, "free": _prepare_free,
            "compact": _prepare_compact}[case["op"]](case, rng, gen)


def _prepare_rows(case, rng, gen):
    ps, hkv, d, dt = case["page_size"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    new, lens = _batch(case, rng)
    table, pages = _page_tables(rng, lens, int(-(-lens.max() // ps)), ps)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    rows = T + case["pads"]
    slots = np.full(rows, -1, np.int32)
    b = np.repeat(np.arange(len(lens)), new)
    pos = (lens - new)[b] + np.arange(T) - start[b]
    slots[:T] = table[b, pos // ps] * ps + pos % ps
    qkv = _keys(gen, (rows, 3 * hkv, d), dt)  # one head group's projection: q, k, v
    return dict(case=case, kv=torch.zeros((pages, hkv, ps * d * 9 // 8), dtype=torch.uint8, device="cuda"),
                k_new=qkv[:, hkv:2 * hkv], v_new=qkv[:, 2 * hkv:], slots=_gpu(slots),
                k_out=torch.empty((rows, hkv, d), dtype=dt, device="cuda"),
                v_out=torch.empty((rows, hkv, d), dtype=dt, device="cuda"))


def _prepare_attend(case, rng, gen):
    ps, hkv, d, dt = case["page_size"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    new, lens = _batch(case, rng)
    table, pages = _page_tables(rng, lens, int(-(-lens.max() // ps)), ps)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    kv = torch.empty((pages, hkv, ps * d * 9 // 8), dtype=torch.uint8, device="cuda")
    _fill_kv4(gen, kv, ps, d)
    q = torch.randn((T, case["q_heads"], d), generator=gen, device="cuda").to(dt)
    return dict(case=case, kv=kv, q=q, table=_gpu(table), seq_lens=_gpu(lens.astype(np.int32)),
                q_start=_gpu(start.astype(np.int32)), longest=int(new.max()), scale=d ** -0.5,
                out=torch.empty_like(q), lse=torch.empty((T, case["q_heads"]), device="cuda"))


def _pools(case, pages, gen):
    """Byte-filled pools of some layers, [pages, bytes of a page]: 4-bit blocks, or K and V in 16 bits."""
    size = _page_bytes(case["pools"], case["page_size"], case["kv_heads"], case["head_dim"])
    each = 1 if case["pools"] == "kv4" else 2
    return [torch.randint(0, 256, (pages, size // each), generator=gen, dtype=torch.uint8, device="cuda")
            for _ in range(each * case["layers"])]


def _prepare_fork(case, rng, gen):
    ps, n, k = case["page_size"], case["parents"], case["children"]
    lens = np.maximum(1, (case["length"] * np.random.default_rng(n + case["length"]).uniform(0.5, 1.0, n))).astype(np.int64)
    lens[0] = case["length"]
    width = int(-(-lens.max() // ps)) + 1
    table, pages = _page_tables(rng, lens, width, ps)
    rows = rng.permutation(n * (k + 1))  # parents and free rows of the table, mixed
    whole = np.full((len(rows), width), -1, np.int32)
    whole[rows[:n]] = table
    all_lens = np.zeros(len(rows), np.int32)
    all_lens[rows[:n]] = lens
    spare = rng.permutation(n * k + 8) + pages
    pages += len(spare)
    return dict(case=case, parents=_gpu(np.repeat(rows[:n], k).astype(np.int32)),
                children=_gpu(rows[n:].astype(np.int32)), table=_gpu(whole), lens=_gpu(all_lens),
                lens_mid=_i32(len(rows)), lens_out=_i32(len(rows)), shares=_i32(pages),
                free_pages=_gpu(np.concatenate([spare, np.full(16, -1)]).astype(np.int32)),
                free_count=_i32(1, len(spare)), free_mid=_i32(1), free_left=_i32(1), copies=_i32((n * k, 2)),
                pools=_pools(case, pages, gen))


def _prepare_free(case, rng, gen):
    ps, B = case["page_size"], case["batch"]
    lens = np.maximum(1, case["length"] * np.random.default_rng(B + case["length"]).uniform(0.4, 1.0, B)).astype(np.int64)
    rng.shuffle(lens)
    width = int(-(-lens.max() // ps)) + 1
    table, pages = _page_tables(rng, lens, width, ps)
    shares = np.zeros(pages, np.int64)
    # some sequences have the first half of another's pages for their own: a prompt in common
    for b in np.nonzero(rng.uniform(size=B) < case["shared"])[0]:
        other = int(rng.integers(0, B))
        common = min(lens[b], lens[other]) // ps // 2
        table[b, :common] = table[other, :common]
    ids, count = np.unique(table[np.arange(width)[None] < (-(-lens // ps))[:, None]], return_counts=True)
    shares[ids] = count - 1
    unused = np.setdiff1d(np.arange(1, pages), ids).astype(np.int32)
    free = np.full(pages, -1, np.int32)
    free[:len(unused)] = rng.permutation(unused)
    return dict(case=case, rows=_gpu(rng.permutation(B)[:case["rows"]].astype(np.int32)), table=_gpu(table),
                lens=_gpu(lens.astype(np.int32)), lens_out=_i32(B), shares=_gpu(shares.astype(np.int32)),
                shares0=_gpu(shares.astype(np.int32)), free_pages=_gpu(free), free_count=_i32(1, len(unused)),
                free_left=_i32(1))


def _prepare_compact(case, rng, gen):
    ps, B, P = case["page_size"], case["batch"], case["pages"]
    n = max(B, int(case["used"] * (P - 1)))
    cut = np.sort(np.random.default_rng(P + B).choice(np.arange(1, n), B - 1, replace=False)) if B > 1 else np.array([], int)
    need = np.diff(np.concatenate([[0], cut, [n]]))
    rng.shuffle(need)
    lens = need * ps - rng.integers(0, ps, B)
    width = int(need.max()) + 1
    ids = rng.permutation(P - 1).astype(np.int32) + 1
    table = np.full((B, width), -1, np.int32)
    table[np.arange(width)[None] < need[:, None]] = ids[:n]
    shares = np.zeros(P, np.int32)
    for b in range(1, B, 3):  # a prompt in common with the sequence before
        common = int(min(need[b], need[b - 1])) // 3
        dropped = table[b, :common].copy()
        table[b, :common] = table[b - 1, :common]
        shares[table[b, :common]] += 1
        ids = np.concatenate([ids, dropped])
    free = np.full(P, -1, np.int32)
    free[:len(ids) - n] = ids[n:]
    st = dict(case=case, table=_gpu(table), lens=_gpu(lens.astype(np.int32)), shares=_gpu(shares), free_pages=_gpu(free),
              free_count=_i32(1, len(ids) - n), moves=_i32((P // 2, 2), -1), n_moves=_i32(1), page_map=_i32(P),
              pools=_pools(case, P, gen))
    st["before"] = [st[x].clone() for x in ("table", "shares", "free_pages")]
    return st


# ----------------------------------------------------------------------------- plain forms: the 4-bit cache
def _parts(pool, ps, d):
    """K codes, V codes [..., page_size, D / 2], K scales, V scales [..., page_size, D / 16] of blocks."""
    h, g = ps * d // 2, ps * d // 16
    cut = (pool[..., :h], pool[..., h:2 * h], pool[..., 2 * h:2 * h + g], pool[..., 2 * h + g:])
    return tuple(x.unflatten(-1, (ps, -1)) for x in cut)


def _quantise(x):
    """Codes in [-7, 7] and scales (a value for 16 elements) of float32 rows."""
    g = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf).unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    t = (top / torch.full_like(top, 7)).clamp(max=MAX_SCALE)  # divided: a number's reciprocal would move a border
    _, e = torch.frexp(t)  # t = m 2^e, m in [1/2, 1): four bits of it are kept
    step = ((e - 4).clamp(min=-17) + 127 << 23).view(torch.float32)  # a power of two
    s = ((t / step).round() * step).clamp(max=MAX_SCALE)
    c = torch.where(s[..., None] > 0, g / s[..., None], 0.0).round().clamp(-7, 7)
    return c.flatten(-2), s


def _scale_byte(s):
    return (s.to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)


def _scale_value(b):
    f = (b.to(torch.int16) << 7).view(torch.float16).float()
    return torch.where(b >= 0xDE, MAX_SCALE, f)


def _packed(c):
    u = (c + 8).to(torch.uint8).unflatten(-1, (-1, 2))
    return u[..., 0] | (u[..., 1] << 4)


def _values(codes, scales):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return (c.unflatten(-1, (-1, 16)) * _scale_value(scales)[..., None]).flatten(-2)


def _plain_rows(st):
    ps, d = st["case"]["page_size"], st["case"]["head_dim"]
    slots, kv = st["slots"].long(), st["kv"]
    on = slots >= 0
    page, row = slots.clamp(min=0) // ps, slots.clamp(min=0) % ps  # page 0 is nobody's
    parts = _parts(kv, ps, d)
    out = []
    for x, codes, scales in ((st["k_new"], parts[0], parts[2]), (st["v_new"], parts[1], parts[3])):
        c, s = _quantise(x.float())
        codes[page, :, row] = torch.where(on[:, None, None], _packed(c), codes[page, :, row])
        scales[page, :, row] = torch.where(on[:, None, None], _scale_byte(s), scales[page, :, row])
        held = _values(codes[page, :, row], scales[page, :, row])
        out.append(torch.where(on[:, None, None], held, 0.0).to(x.dtype))
    return {"k": out[0], "v": out[1]}


def _plain_attend(st):
    case, q, table = st["case"], st["q"], st["table"].long()
    ps, d = case["page_size"], case["head_dim"]
    T, Hq, _ = q.shape
    (B, W), hkv, n = table.shape, case["kv_heads"], st["longest"]
    pages = table.clamp(min=0)
    lens, start = st["seq_lens"].long(), st["q_start"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(n, device=q.device)
    at = (start[:-1, None] + i).clamp(max=T - 1)
    out, lse = torch.empty_like(q), torch.empty_like(st["lse"])
    G = Hq // hkv
    seq = torch.repeat_interleave(torch.arange(B, device=q.device), new, output_size=T)
    mine = torch.arange(T, device=q.device) - start[seq]
    reach = (lens - new)[:, None] + i + 1  # [B, n]
    live = torch.arange(W * ps, device=q.device) < reach[..., None]
    live = live.repeat_interleave(G, 1)  # [B, n G, keys]
    for h in range(hkv):
        kc, vc, ks, vs = _parts(st["kv"][pages, h], ps, d)
        keys, vals = _values(kc, ks).flatten(1, 2), _values(vc, vs).flatten(1, 2)
        g = q[at][:, :, h * G:(h + 1) * G].float().flatten(1, 2)  # [B, n G, d]
        s = torch.where(live, g @ keys.transpose(-1, -2) * st["scale"], -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        w = torch.exp(s - top)
        total = w.sum(-1, keepdim=True)
        o = torch.where(total > 0, (w @ vals) / total, 0.0)
        heads = slice(h * G, (h + 1) * G)
        out[:, heads] = o.view(B, n, G, d)[seq, mine].to(q.dtype)
        lse[:, heads] = (top + torch.log(total)).view(B, n, G)[seq, mine]
    return {"out": out, "lse": lse}


# ----------------------------------------------------------------------------- plain forms: pages
def _plain_copy(pools, pairs):
    src, dst = pairs[:, 0].long(), pairs[:, 1].long()
    for p in pools:
        p[dst] = p[src]


def _plain_free_rows(rows, table, lens, lens_out, shares, free_pages, free_count, free_left, ps):
    r = rows.long()
    W = table.shape[1]
    lens_out.copy_(lens)
    lens_out[r] = 0
    n = (lens[r].long() + ps - 1) // ps
    listed = (torch.arange(W, device=r.device) < n[:, None]).flatten()
    page = torch.where(listed, table[r].long().flatten(), 0)
    released = torch.zeros_like(shares).index_add_(0, page, listed.int())
    gone = released > shares
    order = torch.arange(page.numel(), device=r.device)
    first = torch.full_like(shares, page.numel(), dtype=torch.long).scatter_reduce_(
        0, page, torch.where(listed, order, page.numel()), "amin")
    push = listed & gone[page] & (first[page] == order)
    left = free_count + push.sum()
    at = torch.where(push, left - push.cumsum(0), free_pages.shape[0])  # the first listing ends up on top
    room = torch.cat([free_pages, free_pages.new_empty(1)])
    room[at] = page.int()
    free_pages.copy_(room[:-1])
    free_left.copy_(left)
    shares.copy_(torch.where(gone, 0, shares - released))


def _plain_fork(st):
    ps, table, lens, shares = st["case"]["page_size"], st["table"], st["lens"].long(), st["shares"]
    parent, child = st["parents"].long(), st["children"].long()
    W = table.shape[1]
    n = lens[parent]
    part = (n % ps != 0).long()
    taken = part.cumsum(0)
    fresh = st["free_pages"][(st["free_count"] - taken).long().clamp(min=0)]
    j = torch.arange(W, device=n.device)
    full = j < (n // ps)[:, None]
    rows = table[parent]
    last = (j == (n // ps)[:, None]) & (part > 0)[:, None]
    old = rows.gather(1, (n // ps)[:, None])[:, 0]
    table[child] = torch.where(full, rows, torch.where(last, fresh[:, None], table[child]))
    shares.index_add_(0, torch.where(full, rows, 0).long().flatten(), full.flatten().int())
    st["lens_mid"].copy_(st["lens"])
    st["lens_mid"][child] = n.int()
    st["free_mid"].copy_(st["free_count"] - taken[-1])
    st["copies"].copy_(torch.where((part > 0)[:, None], torch.stack([old, fresh], 1), -1))
    _plain_copy(st["pools"], st["copies"][part > 0])
    _plain_free_rows(st["children"], table, st["lens_mid"], st["lens_out"], shares, st["free_pages"], st["free_mid"],
                     st["free_left"], ps)


def _plain_compact(st):
    ps, table, shares, free, count = (st["case"]["page_size"], st["table"], st["shares"], st["free_pages"],
                                      st["free_count"])
    B, W = table.shape
    P, dev = shares.shape[0], table.device
    listed = torch.arange(W, device=dev) < ((st["lens"].long() + ps - 1) // ps)[:, None]
    page = torch.where(listed, table.long(), P)
    used = torch.zeros(P + 1, dtype=torch.long, device=dev)
    used[page.flatten()] = 1
    used = used[:P]
    idle = torch.zeros(P + 1, dtype=torch.long, device=dev)
    idle[torch.where(torch.arange(P, device=dev) < count, free, P).long()] = 1
    idle = idle[:P]
    below = torch.cat([idle.new_zeros(1), idle.cumsum(0)])  # free pages below x
    above = used.sum() - torch.cat([used.new_zeros(1), used.cumsum(0)])  # used pages at or above x
    x = (below < above).sum()  # the first boundary with as many free pages below as used ones above
    ids = torch.arange(P, device=dev)
    to = (idle > 0) & (ids < x)
    frm = (used > 0) & (ids >= x)
    pairs = torch.full((P + 1, 2), -1, dtype=torch.long, device=dev)
    pairs[torch.where(to, to.cumsum(0) - 1, P), 1] = ids
    pairs[torch.where(frm, frm.cumsum(0) - 1, P), 0] = ids
    pairs = pairs[:int(to.sum())]
    st["n_moves"].fill_(len(pairs))
    st["moves"][:len(pairs)] = pairs.int()
    where = ids.clone()
    where[pairs[:, 0]] = pairs[:, 1]
    st["page_map"].copy_(where)
    table.copy_(torch.where(listed, where[table.clamp(min=0).long()].int(), table))
    shares[pairs[:, 1]] = shares[pairs[:, 0]]
    shares[pairs[:, 0]] = 0
    now = (((idle > 0) & (ids >= x)) | frm).nonzero()[:, 0].flip(0)  # the lowest page on top
    free[:len(now)] = now.int()
    _plain_copy(st["pools"], pairs)


# ----------------------------------------------------------------------------- one pass
FORKED = ("table", "lens_mid", "lens_out", "shares", "free_pages", "free_mid", "free_left", "copies", "pools")
FREED = ("lens_out", "shares", "free_pages", "free_left")
COMPACTED = ("table", "shares", "free_pages", "moves", "n_moves", "page_map", "pools")


def run(st):
    op, ps = st["case"]["op"], st["case"]["page_size"]
    if own:
        import paged_kv_cache_201_gb300 as pa
    if op == "rows":
        if not own:
            return _plain_rows(st)
        pa.paged_attn_append_kv4(st["k_new"], st["v_new"], st["slots"], st["kv"])
        pa.paged_attn_gather_kv4(st["kv"], st["slots"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if op == "attend":
        if not own:
            return _plain_attend(st)
        pa.paged_attn_fwd_kv4(st["q"], st["kv"], st["table"], st["seq_lens"], True, None, st["scale"], st["out"],
                              st["lse"], q_start=st["q_start"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "fork":
        # the children live for a while, then their rows are given back
        if own:
            pa.paged_attn_fork(st["parents"], st["children"], st["table"], st["lens"], st["lens_mid"], st["shares"],
                               st["free_pages"], st["free_count"], st["free_mid"], st["copies"], ps)
            pa.paged_attn_copy_pages(st["pools"], st["copies"])
            pa.paged_attn_free(st["children"], st["table"], st["lens_mid"], st["lens_out"], st["shares"],
                               st["free_pages"], st["free_mid"], st["free_left"], ps)
        else:
            _plain_fork(st)
        return {k: st[k] for k in FORKED}
    if op == "free":
        st["shares"].copy_(st["shares0"])  # the sequences are there again
        (pa.paged_attn_free if own else _plain_free_rows)(
            st["rows"], st["table"], st["lens"], st["lens_out"], st["shares"], st["free_pages"], st["free_count"],
            st["free_left"], ps)
        return {k: st[k] for k in FREED}
    for x, old in zip(("table", "shares", "free_pages"), st["before"]):  # the pool is scattered again
        st[x].copy_(old)
    if own:
        pa.paged_attn_compact(st["table"], st["lens"], st["shares"], st["free_pages"], st["free_count"], st["moves"],
                              st["n_moves"], st["page_map"], ps)
        pa.paged_attn_copy_pages(st["pools"], st["moves"], st["n_moves"])
    else:
        _plain_compact(st)
    return {k: st[k] for k in COMPACTED}


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, ps = case["op"], case["page_size"]
    if op == "free":
        entries = case["rows"] * 0.7 * case["length"] / ps
        return {"bytes": entries * (4 + 8 + 4 * (1 - case["shared"] / 2)) + 4.0 * case["rows"] + 8.0 * case["batch"],
                "flops": 0}
    if op == "fork":
        n, block = case["parents"] * case["children"], _page_bytes(case["pools"], ps, case["kv_heads"], case["head_dim"])
        entries = n * (0.75 * case["length"] / ps if case["parents"] > 1 else case["length"] / ps)
        # table rows read and written, shares counted up and down, last pages copied, rows read to be freed
        return {"bytes": entries * (8 + 16 + 4) + 2.0 * n * case["layers"] * block, "flops": 0}
    if op == "compact":
        P, used = case["pages"], case["used"]
        block = _page_bytes(case["pools"], ps, case["kv_heads"], case["head_dim"])
        moves = P * used * (1 - used)
        return {"bytes": 4.0 * P * (2 * used + 1 + 2 * (1 - used)) + 16.0 * moves + 2.0 * moves * case["layers"] * block,
                "flops": 0}
    B, hkv, d, e, chunk = case["batch"], case["kv_heads"], case["head_dim"], ESIZE[case["dtype"]], case["chunk"]
    T = B if chunk == 1 else chunk + (B - 1) * 0.75 * chunk
    if op == "rows":
        return {"bytes": 4.0 * T * hkv * d * e + 2 * T * hkv * d * 9 / 8 + 8.0 * T, "flops": 0}
    mean_len = max(chunk, case["length"] * (1 + 0.7 * (B - 1)) / B)
    Hq = case["q_heads"]
    return {"bytes": B * mean_len * hkv * d * 9 / 8 + 2.0 * T * Hq * d * e + 4.0 * T * Hq,
            "flops": 4.0 * T * Hq * d * (mean_len - (chunk - 1) / 2)}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _held64(x):
    """The values that 4 bits hold of rows x [..., D], from the tables of all scales and all codes."""
    byte = np.arange(0xDF)
    scales = np.where(byte < 8, byte * 2.0 ** -17, (8 + byte % 8) * 2.0 ** (byte // 8 - 18.0))
    g = x.reshape(*x.shape[:-1], -1, 16)
    t = np.abs(g).max(-1) / 7
    i = np.clip(np.searchsorted(scales, t, side="right") - 1, 0, len(scales) - 2)
    up, down = scales[i + 1] - t, t - scales[i]
    i = i + ((up < down) | ((up == down) & (i % 2 == 1)))
    s = scales[i][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.clip(np.rint(g / s), -7, 7), 0.0)
    return (c * s).reshape(x.shape)


def _exact_rows(st):
    on = (st["slots"] >= 0).cpu().numpy()[:, None, None]
    return {n: torch.from_numpy(np.where(on, _held64(st[n + "_new"].double().cpu().numpy()), 0.0)) for n in "kv"}


def _exact_attend(st):
    case, q, table, lens, starts = st["case"], st["q"], st["table"].long(), st["seq_lens"].tolist(), st["q_start"].tolist()
    ps, d, hkv = case["page_size"], case["head_dim"], case["kv_heads"]
    G = case["q_heads"] // hkv
    half, few = ps * d // 2, ps * d // 16
    byte = np.arange(256).clip(max=0xDE)
    scale_of = _gpu(np.where(byte < 8, byte * 2.0 ** -17, (8 + byte % 8) * 2.0 ** (byte // 8 - 18.0)))
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(len(lens)):
        n, L = starts[b + 1] - starts[b], lens[b]
        blocks = st["kv"][table[b, :-(-L // ps)]]
        for h in range(hkv):
            rows = []
            for at, sc in ((0, 2 * half), (half, 2 * half + few)):
                codes = blocks[:, h, at:at + half].reshape(-1, d // 2).to(torch.int64)
                c = torch.empty(codes.shape[0], d, dtype=torch.float64, device=q.device)
                c[:, 0::2], c[:, 1::2] = (codes % 16 - 8).double(), (codes // 16 - 8).double()
                s = scale_of[blocks[:, h, sc:sc + few].reshape(-1, d // 16).long()]
                rows.append((c * s.repeat_interleave(16, 1))[:L])
            step = max(1, (1 << 25) // max(1, L * G))
            for t0 in range(starts[b], starts[b + 1], step):
                t1 = min(t0 + step, starts[b + 1])
                reach = L - starts[b + 1] + torch.arange(t0, t1, device=q.device) + 1
                heads = slice(h * G, (h + 1) * G)
                s = torch.einsum("tgd,kd->tgk", q[t0:t1, heads].double(), rows[0]) * st["scale"]
                s.masked_fill_((torch.arange(L, device=q.device) >= reach[:, None])[:, None], -math.inf)
                total = torch.logsumexp(s, -1)
                out[t0:t1, heads] = torch.einsum("tgk,kd->tgd", torch.exp(s - total[..., None]), rows[1])
                lse[t0:t1, heads] = total
    return {"out": out, "lse": lse}


def _free_list(rows, table, lens, shares, stack, ps):
    """Sequences given up one after the other, the last first, each from its last page: changes its lists."""
    for r in reversed(rows):
        for j in range(-(-lens[r] // ps) - 1, -1, -1):
            p = table[r][j]
            if shares[p] == 0:
                stack.append(p)
            else:
                shares[p] -= 1
        lens[r] = 0


def _int(x):
    return torch.tensor(x, dtype=torch.int32)


def _padded(stack, old):
    return _int(stack + old[len(stack):])


def _exact_fork(st):
    ps, table, lens, shares = st["case"]["page_size"], st["table"].tolist(), st["lens"].tolist(), st["shares"].tolist()
    old = st["free_pages"].tolist()
    stack, copies, pools = old[:int(st["free_count"])], [], st["pools"]
    for a, b in zip(st["parents"].tolist(), st["children"].tolist()):
        for j in range(lens[a] // ps):
            table[b][j] = table[a][j]
            shares[table[a][j]] += 1
        copies.append([-1, -1])
        if lens[a] % ps:
            copies[-1] = [table[a][lens[a] // ps], stack.pop()]
            table[b][lens[a] // ps] = copies[-1][1]
            for p in pools:
                p[copies[-1][1]] = p[copies[-1][0]]
        lens[b] = lens[a]
    mid, left = list(lens), len(stack)
    _free_list(st["children"].tolist(), table, lens, shares, stack, ps)
    return {"table": _int(table), "lens_mid": _int(mid), "lens_out": _int(lens), "shares": _int(shares),
            "free_pages": _padded(stack, old), "free_mid": _int([left]), "free_left": _int([len(stack)]),
            "copies": _int(copies), "pools": pools}


def _exact_free(st):
    table, lens, shares = st["table"].tolist(), st["lens"].tolist(), st["shares"].tolist()
    old = st["free_pages"].tolist()
    stack = old[:int(st["free_count"])]
    _free_list(st["rows"].tolist(), table, lens, shares, stack, st["case"]["page_size"])
    return {"lens_out": _int(lens), "shares": _int(shares), "free_pages": _padded(stack, old),
            "free_left": _int([len(stack)])}


def _exact_compact(st):
    ps, table, lens, shares = st["case"]["page_size"], st["table"].tolist(), st["lens"].tolist(), st["shares"].tolist()
    old = st["free_pages"].tolist()
    stack = old[:int(st["free_count"])]
    used = sorted({p for r, n in zip(table, lens) for p in r[:-(-n // ps)]})
    idle = sorted(stack)
    k = 0  # the k highest used pages go to the k lowest free ones as long as that is downwards
    while k < min(len(used), len(idle)) and idle[k] < used[-1 - k]:
        k += 1
    pairs = list(zip(used[len(used) - k:], idle[:k]))
    where = list(range(len(shares)))
    for a, b in pairs:
        where[a] = b
        shares[b], shares[a] = shares[a], 0
        for p in st["pools"]:
            p[b] = p[a]
    for r, n in zip(table, lens):
        for j in range(-(-n // ps)):
            r[j] = where[r[j]]
    now = sorted(idle[k:] + [a for a, _ in pairs], reverse=True)
    moves = st["moves"].tolist()
    moves[:k] = [list(m) for m in pairs]
    return {"table": _int(table), "shares": _int(shares), "free_pages": _padded(now, old), "moves": _int(moves),
            "n_moves": _int([k]), "page_map": _int(where), "pools": st["pools"]}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rows": _exact_rows, "attend": _exact_attend, "fork": _exact_fork, "free": _exact_free,
            "compact": _exact_compact}[case["op"]](st)
