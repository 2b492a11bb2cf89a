"""Cases of the page-sparse serving operators: tables and slots, append, page selection, sparse attention.

One serving step over the paged K/V cache runs them in this order: ``paged_attn_step_tables`` turns the
requests' lengths into block tables and slots, ``paged_attn_append`` writes the new tokens' K and V rows
and the envelopes (corner values) of the pages they land in, ``paged_attn_select_pages`` picks the pages
each token attends to by a cheap score, and ``paged_attn_fwd_sparse`` attends over them.

``own`` selects what ``run`` computes: the operators' plain form (elementary torch operations) or the
library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a small server's decode step: one new token for each of 16 requests
        dict(name="tables_decode_16", op="tables", batch=16, capacity=16, width=128, page_size=16, chunk=1,
             free=256),
        # a large scheduler step: 1024 requests, some of them prefill chunks of up to 2048 tokens
        dict(name="tables_mixed_1024", op="tables", batch=1024, capacity=65536, width=512, page_size=16, chunk=2048,
             free=8192),
        # one decode step's K and V rows of 256 sequences (8 kv heads of 128), a few rows of padding
        dict(name="append_decode_256", op="append", batch=256, chunk=1, pads=5, kv_heads=8, head_dim=128, page_size=16,
             length=512, dtype="bf16"),
        # prefill chunks of 8192 tokens in all, in large pages, their K and V sliced out of a QKV projection
        dict(name="append_chunk_8192", op="append", batch=4, chunk=2048, pads=0, kv_heads=8, head_dim=128, page_size=64,
             length=8192, dtype="f16"),
        # a verification step of a few tokens for each sequence, in float32 with an odd head count
        dict(name="append_f32_odd", op="append", batch=7, chunk=5, pads=1, kv_heads=3, head_dim=256, page_size=32,
             length=300, dtype="f32"),
        # decode of 256 ragged sequences of up to 4096 tokens: 32 of up to 256 pages each
        dict(name="select_decode_256", op="select", batch=256, chunk=1, q_heads=32, kv_heads=8, head_dim=128,
             page_size=16, length=4096, top_k=32, sink=1, local=2, dtype="bf16"),
        # two very long contexts, one new token each: few rows, a long axis
        dict(name="select_long_2", op="select", batch=2, chunk=1, q_heads=64, kv_heads=4, head_dim=128, page_size=32,
             length=131072, top_k=64, sink=1, local=4, dtype="f16"),
        # prefill chunks of 512 tokens behind long prefixes: every token picks its own pages
        dict(name="select_chunk_1024", op="select", batch=2, chunk=512, q_heads=32, kv_heads=8, head_dim=128,
             page_size=16, length=8192, top_k=64, sink=1, local=4, dtype="bf16"),
        # decode of 256 sequences over 64 listed pages each
        dict(name="attend_decode_256", op="attend", batch=256, chunk=1, q_heads=32, kv_heads=8, head_dim=128,
             page_size=16, length=4096, top_k=64, dtype="bf16"),
        # one very long context: 8 rows of units, 128 pages each
        dict(name="attend_long_1", op="attend", batch=1, chunk=1, q_heads=32, kv_heads=8, head_dim=128, page_size=32,
             length=131072, top_k=128, dtype="bf16"),
        # the same prefill chunks as above: every token has its own list
        dict(name="attend_chunk_1024", op="attend", batch=2, chunk=512, q_heads=32, kv_heads=8, head_dim=128,
             page_size=16, length=8192, top_k=64, dtype="f16"),
        # a few tokens each in float32, three heads to a group, lists that reach past short sequences
        dict(name="attend_f32_odd", op="attend", batch=5, chunk=3, q_heads=6, kv_heads=2, head_dim=64, page_size=16,
             length=200, top_k=9, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "append", "select", "select", "attend", "attend"])
    ps = rng.choice([16, 32, 64])
    if op == "tables":
        batch = _log_int(rng, 1, 1024)
        chunk = rng.choice([1, _log_int(rng, 2, 2048)])
        capacity = min(65536, batch * max(1, chunk // rng.randint(1, 8)))
        return dict(op=op, batch=batch, capacity=capacity, width=_log_int(rng, 40, 512), page_size=ps, chunk=chunk,
                    free=_log_int(rng, 16, 8192))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    head_dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "append":
        batch = _log_int(rng, 1, 512)
        chunk = rng.choice([1, _log_int(rng, 2, 2048)])
        while batch * chunk * hkv * head_dim * ESIZE[dtype] > 8192 * 8 * 128 * 2:
            batch, chunk = max(1, batch // 2), max(1, (chunk * 2) // 3)
        length = max(chunk + 1, min(_log_int(rng, 64, 16384), (1 << 27) // (batch * hkv * head_dim)))
        return dict(op=op, batch=batch, chunk=chunk, pads=rng.choice([0, 0, rng.randint(1, 9)]), kv_heads=hkv,
                    head_dim=head_dim, page_size=ps, length=length, dtype=dtype)
    group = rng.choice([1, 2, 3, 4, 7, 8, 16, 24])
    batch = _log_int(rng, 1, 256)
    chunk = rng.choice([1, 1, _log_int(rng, 2, 512)])
    length = max(chunk, _log_int(rng, 33, 131072))
    top_k = _log_int(rng, 4, 160)
    if op == "select":
        def cost():
            pages = -(-length // ps)
            return max(batch * pages * hkv * head_dim / (256 * 256 * 8 * 128),
                       batch * chunk * pages * hkv * group * head_dim / (1024 * 512 * 32 * 128))
        while cost() > 1:
            batch, chunk, length = max(1, batch * 2 // 3), max(1, chunk * 2 // 3), max(chunk, length * 3 // 4)
        return dict(op=op, batch=batch, chunk=chunk, q_heads=group * hkv, kv_heads=hkv, head_dim=head_dim, page_size=ps,
                    length=length, top_k=top_k, sink=rng.randint(0, 1), local=rng.randint(0, 3), dtype=dtype)

    def cost():
        return max(batch * chunk * hkv * top_k * ps * head_dim * ESIZE[dtype] / (1024 * 8 * 1024 * 128 * 2),
                   batch * length * hkv * head_dim * ESIZE[dtype] / (256 * 4096 * 8 * 128 * 2))
    while cost() > 1:
        batch, chunk, length = max(1, batch * 2 // 3), max(1, chunk * 2 // 3), max(chunk, length * 3 // 4)
        top_k = max(4, top_k * 4 // 5)
    return dict(op=op, batch=batch, chunk=chunk, q_heads=group * hkv, kv_heads=hkv, head_dim=head_dim, page_size=ps,
                length=length, top_k=top_k, dtype=dtype)


# ----------------------------------------------------------------------------- inputs
def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


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


def _kv_pools(gen, pages, case):
    shape, dt = (pages, case["page_size"], case["kv_heads"], case["head_dim"]), DTYPES[case["dtype"]]
    k = torch.empty(shape, dtype=dt, device="cuda")
    v = torch.empty(shape, dtype=dt, device="cuda")
    for pool in (k, v):
        for part in pool.split(max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))):
            part.copy_(_keys(gen, part.shape, dt))
    return k, v


def prepare(case, seed):
    rng = np.random.default_rng([seed, 71])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ps, op = case["page_size"], case["op"]
    st = {"case": case}
    if op == "tables":
        B, W = case["batch"], case["width"]
        kind = rng.uniform(size=B)
        chunk = np.exp(rng.uniform(0, math.log(case["chunk"] + 1), B)).astype(np.int64).clip(1, case["chunk"])
        new = np.where(kind < 0.85, 1, np.where(kind < 0.95, chunk, 0))  # decode, prefill chunk, idle
        cached = np.minimum(rng.integers(0, W * ps, B), np.maximum(W * ps - new, 0))
        cached[rng.uniform(size=B) < 0.05] = 0
        need = -(-cached // ps)
        pool = int(need.sum()) + case["free"] + 1
        ids = rng.permutation(pool - 1).astype(np.int32) + 1
        table = np.full((B, W), -1, np.int32)
        table[np.arange(W)[None] < need[:, None]] = ids[:int(need.sum())]
        i32 = dict(dtype=torch.int32, device="cuda")
        st |= dict(cached=_gpu(cached.astype(np.int32)), new=_gpu(new.astype(np.int32)),
                   free_pages=_gpu(ids[int(need.sum()):]), free_count=torch.full((1,), case["free"], **i32),
                   table=_gpu(table), num_pages=pool, seq_lens=torch.empty(B, **i32), q_offset=torch.empty(B, **i32),
                   q_start=torch.empty(B + 1, **i32), slots=torch.empty(case["capacity"], **i32),
                   free_left=torch.empty(1, **i32))
        return st
    new, lens = _batch(case, rng)
    B, Hkv, D = case["batch"], case["kv_heads"], case["head_dim"]
    width = int(-(-lens.max() // ps))
    table, pages = _page_tables(rng, lens, width, ps)
    q_start = np.concatenate([[0], np.cumsum(new)])
    T = int(q_start[-1])
    if op == "append":
        rows = T + case["pads"]
        slots = np.full(rows, -1, np.int32)
        b = np.repeat(np.arange(B), new)
        pos = (lens - new)[b] + np.arange(T) - q_start[b]
        slots[:T] = table[b, pos // ps] * ps + pos % ps
        k, v = _kv_pools(gen, pages, case)
        qkv = _keys(gen, (rows, 3 * Hkv, D), DTYPES[case["dtype"]])  # one head group's projection: q, k, v
        env = torch.zeros(pages, Hkv, 2, D, dtype=torch.int8, device="cuda")
        st |= dict(k=k, v=v, k_new=qkv[:, Hkv:2 * Hkv], v_new=qkv[:, 2 * Hkv:], slots=_gpu(slots), env=env,
                   env_scale=torch.zeros(pages, Hkv, device="cuda"), touched=len(np.unique(slots[:T] // ps)))
        return st
    st |= dict(q=torch.randn((T, case["q_heads"], D), generator=gen, device="cuda").to(DTYPES[case["dtype"]]),
               table=_gpu(table), seq_lens=_gpu(lens.astype(np.int32)), q_start=_gpu(q_start.astype(np.int32)),
               longest=int(new.max()), sel=torch.empty(T, Hkv, case["top_k"], dtype=torch.int32, device="cuda"))
    if op == "select":
        # envelopes of correlated pages, quantised as the append leaves them
        mid = torch.randn((pages, Hkv, D), generator=gen, device="cuda")
        half = torch.rand((pages, Hkv, D), generator=gen, device="cuda") * 1.5 + 0.2
        lo, hi = mid - half, mid + half
        top = torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True)
        st |= dict(env=torch.stack([(lo / top * 127).round(), (hi / top * 127).round()], 2).to(torch.int8),
                   env_scale=(top / 127)[..., 0].contiguous())
        return st
    # the lists that a selection gives: distinct reachable pages in ascending order, -1 behind them
    b = np.repeat(np.arange(B), new)
    reach = _gpu((lens - new)[b] + np.arange(T) - q_start[b] + 1)
    n_pages = (reach + ps - 1) // ps
    score = torch.rand((T, Hkv, width), generator=gen, device="cuda")
    page = torch.arange(width, device="cuda")
    score += 2.0 * ((page == 0) | (page + 2 >= n_pages[:, None]))[:, None]
    score = torch.where((page < n_pages[:, None])[:, None], score, -1.0)
    top = torch.topk(score, min(case["top_k"], width), dim=-1)
    idx = torch.where(top.values < 0, width, top.indices).sort(-1).values
    st["sel"].fill_(-1)
    st["sel"][..., :idx.shape[-1]] = torch.where(idx == width, -1, idx).to(torch.int32)
    k, v = _kv_pools(gen, pages, case)
    st |= dict(k=k, v=v, scale=D ** -0.5, out=torch.empty_like(st["q"]),
               lse=torch.empty(T, case["q_heads"], device="cuda"))
    return st


# ----------------------------------------------------------------------------- plain forms
def _plain_tables(st):
    ps, T = st["case"]["page_size"], st["case"]["capacity"]
    c, n, f, table = st["cached"].long(), st["new"].long(), st["free_count"].long(), st["table"]
    W = table.shape[1]
    have, want = (c + ps - 1) // ps, (c + n + ps - 1) // ps
    usable = (c >= 0) & (n >= 0) & (want <= W)
    need = torch.where(usable, want - have, 0)
    tok = torch.where(usable, n, 0)
    served = usable & ((need == 0) | (need.cumsum(0) <= f)) & (tok.cumsum(0) <= T)
    need, tok = torch.where(served, need, 0), torch.where(served, tok, 0)
    first_page = need.cumsum(0) - need
    ends = tok.cumsum(0)
    q_start = torch.cat([torch.zeros_like(ends[:1]), ends])
    page = torch.arange(W, device=c.device)
    at = f - 1 - (first_page[:, None] + page - have[:, None])
    fresh = (page >= have[:, None]) & (page < (have + need)[:, None])
    ids = st["free_pages"][at.clamp(0, st["free_pages"].shape[0] - 1)]
    table.copy_(torch.where(fresh, ids, table))
    t = torch.arange(T, device=c.device)
    b = torch.searchsorted(ends, t, right=True).clamp(max=c.shape[0] - 1)
    pos = c[b] + t - q_start[b]
    slots = table[b, (pos // ps).clamp(0, W - 1)].long() * ps + pos % ps
    slots = torch.where(t < ends[-1], slots, -1)
    return {"table": table, "seq_lens": (c + tok).int(), "q_offset": c.int(), "q_start": q_start.int(),
            "slots": slots.int(), "free_left": (f - need.sum()).int()}


def _plain_append(st):
    k, v, slots = st["k"], st["v"], st["slots"].long()
    P, ps, Hkv, D = k.shape
    on = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)  # page 0 is nobody's: what has no slot leaves its first row as it is
    for_k, for_v = k.view(P * ps, Hkv, D), v.view(P * ps, Hkv, D)
    for_k[at] = torch.where(on, st["k_new"], for_k[at])
    for_v[at] = torch.where(on, st["v_new"], for_v[at])
    # the last new token of each page closes it: the envelope runs over the rows up to there
    nxt = torch.cat([slots[1:], slots.new_full((1,), -1)])
    last = (slots >= 0) & (nxt != slots + 1) | (slots >= 0) & (slots % ps == ps - 1)
    t = torch.argsort(last.to(torch.int8), descending=True, stable=True)[:st["touched"]]
    page, row = slots[t] // ps, slots[t] % ps
    rows = k[page].float()
    live = (torch.arange(ps, device=k.device) <= row[:, None])[:, :, None, None]
    lo = torch.where(live, rows, math.inf).amin(1)
    hi = torch.where(live, rows, -math.inf).amax(1)
    top = torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True)
    corner = torch.stack([lo, hi], 2)
    part = torch.where(top[..., None] > 0, corner / top[..., None], 0.0)
    st["env"][page] = (part * 127).round().to(torch.int8)
    st["env_scale"][page] = top[..., 0] / 127
    return {"k": k, "v": v, "env": st["env"], "env_scale": st["env_scale"]}


def _token_rows(st):
    """(sequence of each packed token, its index there, keys that it reaches)"""
    q_start = st["q_start"].long()
    t = torch.arange(st["q"].shape[0], device=q_start.device)
    b = torch.searchsorted(q_start[1:], t, right=True)
    i = t - q_start[b]
    new = q_start[1:] - q_start[:-1]
    return b, i, (st["seq_lens"].long() - new)[b] + i + 1


def _plain_select(st):
    case, q, env, table = st["case"], st["q"], st["env"], st["table"].long()
    ps, K = case["page_size"], case["top_k"]
    T, Hq, D = q.shape
    Hkv, (B, W) = env.shape[1], table.shape
    n = st["longest"]
    at = (st["q_start"][:-1].long()[:, None] + torch.arange(n, device=q.device)).clamp(max=T - 1)
    g = q[at].float().view(B, n, Hkv, Hq // Hkv, D).transpose(1, 2)  # padded to the longest sequence
    top = g.abs().amax((-2, -1), keepdim=True)
    qi = torch.where(top > 0, g / top, 0.0).mul(127).round()
    both = torch.cat([qi.clamp(max=0), qi.clamp(min=0)], -1).reshape(B, Hkv, -1, 2 * D)
    pages = table.clamp(min=0)
    corners = env[pages].permute(0, 2, 3, 4, 1).reshape(B, Hkv, 2 * D, W).float()
    whole = (both @ corners).view(B, Hkv, n, Hq // Hkv, W).amax(3)  # integers below 2^24: exact
    scale = st["env_scale"][pages].transpose(1, 2)[:, :, None]
    score = torch.where(scale.isinf(), math.inf, whole * scale)
    b, i, reach = _token_rows(st)
    score = score.transpose(1, 2)[b, i].double()  # [T, Hkv, W]
    n_pages = ((reach + ps - 1) // ps)[:, None, None]
    page = torch.arange(W, device=q.device)
    forced = (page < case["sink"]) | (page >= n_pages - case["local"])
    score = torch.where(forced, 1e300, score.clamp(-1e200, 1e200))
    score = torch.where(page < n_pages, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)
    idx = torch.where(best.values[..., :K] == -math.inf, W, best.indices[..., :K]).sort(-1).values
    sel = torch.full((T, Hkv, K), -1, dtype=torch.int32, device=q.device)
    sel[..., :idx.shape[-1]] = torch.where(idx == W, -1, idx)
    return sel


def _plain_attend(st):
    q, k, v, sel = st["q"], st["k"], st["v"], st["sel"].long()
    T, Hq, D = q.shape
    ps, Hkv = k.shape[1], k.shape[2]
    b, _, reach = _token_rows(st)
    pages = st["table"].long()[b[:, None, None], sel.clamp(min=0)].clamp(min=0)
    head = torch.arange(Hkv, device=q.device)[:, None]
    keys = k.transpose(1, 2)[pages, head].float().view(T, Hkv, -1, D)
    vals = v.transpose(1, 2)[pages, head].float().view(T, Hkv, -1, D)
    pos = sel[..., None] * ps + torch.arange(ps, device=q.device)
    live = ((sel >= 0)[..., None] & (pos < reach[:, None, None, None])).view(T, Hkv, 1, -1)
    s = q.float().view(T, Hkv, Hq // Hkv, D) @ keys.transpose(-1, -2) * st["scale"]
    s = torch.where(live, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(s - top)
    total = w.sum(-1, keepdim=True)
    out = torch.where(total > 0, (w @ torch.where(live.transpose(-1, -2), vals, 0.0)) / total, 0.0)
    return {"out": out.view(T, Hq, D).to(q.dtype), "lse": (top + torch.log(total)).view(T, Hq)}


# ----------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        import paged_kv_cache_201_gb300 as pa
        if op == "tables":
            pa.paged_attn_step_tables(st["cached"], st["new"], st["free_pages"], st["free_count"], st["table"],
                                      st["seq_lens"], st["q_offset"], st["q_start"], st["slots"], st["free_left"],
                                      st["case"]["page_size"], st["num_pages"])
            return {n: st[n] for n in ("table", "seq_lens", "q_offset", "q_start", "slots", "free_left")}
        if op == "append":
            pa.paged_attn_append(st["k_new"], st["v_new"], st["slots"], st["k"], st["v"], st["env"], st["env_scale"])
            return {n: st[n] for n in ("k", "v", "env", "env_scale")}
        if op == "select":
            pa.paged_attn_select_pages(st["q"], st["env"], st["env_scale"], st["table"], st["seq_lens"], True, None,
                                       st["case"]["sink"], st["case"]["local"], st["sel"], st["case"]["page_size"],
                                       q_start=st["q_start"])
            return st["sel"]
        pa.paged_attn_fwd_sparse(st["q"], st["k"], st["v"], st["table"], st["seq_lens"], True, None, st["sel"],
                                 st["scale"], st["out"], st["lse"], q_start=st["q_start"])
        return {"out": st["out"], "lse": st["lse"]}
    plain = {"tables": _plain_tables, "append": _plain_append, "select": _plain_select, "attend": _plain_attend}
    return plain[op](st)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, ps, B = case["op"], case["page_size"], case["batch"]
    if op == "tables":
        # the lengths in, four arrays of the batch out, the slots, and each new page's id read and written
        mean_new = 0.85 + 0.1 * max(1.0, (case["chunk"] - 1) / math.log(case["chunk"] + 1))
        tokens = min(case["capacity"], B * mean_new)
        return {"bytes": 4.0 * (2 * B + 3 * B + case["capacity"]) + 8.0 * min(case["free"], tokens / ps + 1),
                "flops": 0}
    e, Hkv, D, chunk = ESIZE[case["dtype"]], case["kv_heads"], case["head_dim"], case["chunk"]
    T = B * chunk if chunk == 1 else chunk + (B - 1) * 0.75 * chunk
    mean_len = case["length"] * (1 + 0.7 * (B - 1)) / B
    if op == "append":
        touched = B * max(1.0, T / B / ps + (0.5 if chunk > 1 else 0))
        old = B * (ps - 1) / 2  # rows already in the first page of each sequence
        return {"bytes": 4.0 * T * Hkv * D * e + old * Hkv * D * e + touched * Hkv * (2 * D + 4) + 4.0 * T, "flops": 0}
    Hq, K = case["q_heads"], case["top_k"]
    if op == "select":
        pages = B * mean_len / ps
        return {"bytes": T * Hq * D * e + pages * (Hkv * (2 * D + 4) + 4) + 4.0 * T * Hkv * K,
                "flops": 4.0 * T * Hq * D * mean_len / ps}
    listed_keys = min(K * ps, mean_len)
    distinct = min(T * K, B * mean_len / ps) if chunk > 1 else B * listed_keys / ps
    return {"bytes": 2.0 * distinct * ps * Hkv * D * e + 2.0 * T * Hq * D * e + 4.0 * T * (Hkv * K + Hq),
            "flops": 4.0 * T * Hq * D * listed_keys}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def _exact_tables(st):
    ps, cap = st["case"]["page_size"], st["case"]["capacity"]
    c, n, stack = st["cached"].tolist(), st["new"].tolist(), st["free_pages"].tolist()
    left, table = int(st["free_count"]), st["table"].cpu().numpy().copy()
    count, pages_asked, tokens_asked, taken = left, 0, 0, 0
    lens, starts, slots = [], [0], []
    for b in range(len(c)):
        have, want = -(-c[b] // ps), -(-(c[b] + n[b]) // ps)
        ok = c[b] >= 0 and n[b] >= 0 and want <= table.shape[1]
        if ok:
            pages_asked, tokens_asked = pages_asked + want - have, tokens_asked + n[b]
            ok = (want == have or pages_asked <= count) and tokens_asked <= cap
        if ok:
            for p in range(have, want):
                table[b, p] = stack[count - 1 - taken]
                taken += 1
            slots += [int(table[b, x // ps]) * ps + x % ps for x in range(c[b], c[b] + n[b])]
        lens.append(c[b] + (n[b] if ok else 0))
        starts.append(len(slots))
    slots += [-1] * (cap - len(slots))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"table": torch.from_numpy(table), "seq_lens": i32(lens), "q_offset": i32(c), "q_start": i32(starts),
            "slots": i32(slots), "free_left": i32([count - taken])}


def _exact_append(st):
    slots = [s for s in st["slots"].tolist()]
    k, v, scale = st["k"].double(), st["v"].double(), st["env_scale"].double()
    P, ps, Hkv, D = k.shape
    t = [i for i, s in enumerate(slots) if s >= 0]
    at = torch.tensor([slots[i] for i in t], device=k.device)
    k.view(-1, Hkv, D)[at] = st["k_new"][t].double()
    v.view(-1, Hkv, D)[at] = st["v_new"][t].double()
    end = {}
    for i in t:
        end[slots[i] // ps] = max(end.get(slots[i] // ps, -1), slots[i] % ps)
    page = torch.tensor(list(end), device=k.device)
    row = torch.tensor(list(end.values()), device=k.device)
    dead = torch.arange(ps, device=k.device)[None] > row[:, None]
    scale[page] = k[page].abs().masked_fill(dead[..., None, None], 0).amax((1, 3)) / 127
    return {"k": k, "v": v, "env": None, "env_scale": scale}


def _exact_attend(st):
    q, table, lens, starts = st["q"], st["table"].long(), st["seq_lens"].tolist(), st["q_start"].tolist()
    T, Hq, D = q.shape
    k, v, sel = st["k"], st["v"], st["sel"].long()
    ps, Hkv = k.shape[1], k.shape[2]
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    step = max(1, (1 << 26) // (sel.shape[-1] * ps * D))
    for b in range(len(lens)):
        for t0 in range(starts[b], starts[b + 1], step):
            t1 = min(t0 + step, starts[b + 1])
            reach = lens[b] - starts[b + 1] + torch.arange(t0, t1, device=q.device) + 1
            for h in range(Hkv):
                j = sel[t0:t1, h]
                pos = (j[..., None] * ps + torch.arange(ps, device=q.device)).flatten(1)
                off = (pos < 0) | (pos >= reach[:, None])
                rows = table[b][j.clamp(min=0)].clamp(min=0)
                kk, vv = (x[rows, :, h].flatten(1, 2).double() for x in (k, v))
                qq = q[t0:t1].view(t1 - t0, Hkv, -1, D)[:, h].double()
                s = torch.einsum("tgd,tkd->tgk", qq, kk) * st["scale"]
                s.masked_fill_(off[:, None], -math.inf)
                total = torch.logsumexp(s, -1)
                w = torch.exp(s - total.nan_to_num(neginf=0.0)[..., None])
                g = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                out[t0:t1, g] = torch.einsum("tgk,tkd->tgd", w, vv.masked_fill(off[..., None], 0))
                lse[t0:t1, g] = total
    return {"out": out, "lse": lse}


def _exact_select(st):
    case, q = st["case"], st["q"]
    ps, K = case["page_size"], case["top_k"]
    T, Hq, D = q.shape
    Hkv = st["env"].shape[1]
    lens, starts, sel = st["seq_lens"].tolist(), st["q_start"].tolist(), []
    group = q.float().view(T, Hkv, -1, D)
    top = group.abs().flatten(2).max(-1).values[..., None, None]
    qi = torch.round(group / top.masked_fill(top == 0, 1) * 127).double()
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        pages = st["table"][b, :-(-lens[b] // ps)].long()
        env = st["env"][pages].double()
        lo, hi = env[:, :, 0], env[:, :, 1]
        x = qi[starts[b]:starts[b + 1]]
        s = torch.einsum("thgd,whd->thgw", x.clamp(min=0), hi) + torch.einsum("thgd,whd->thgw", x.clamp(max=0), lo)
        s = s.max(2).values.float() * st["env_scale"][pages].T[None]
        s = s.masked_fill(st["env_scale"][pages].T[None].isinf(), math.inf)
        for i in range(n):
            count = (lens[b] - n + i + ps) // ps
            order = torch.sort(s[i, :, :count], dim=-1, descending=True, stable=True).indices
            place = torch.empty_like(order).scatter_(1, order, torch.arange(count, device=q.device).expand(Hkv, -1))
            place[:, :case["sink"]] -= 1 << 30
            place[:, max(0, count - case["local"]):] -= 1 << 30
            keep = place.argsort(-1)[:, :K].sort(-1).values
            sel.append(torch.nn.functional.pad(keep, (0, K - keep.shape[1]), value=-1))
    return torch.stack(sel).int()


def exact(case, seed):
    st = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "select": _exact_select,
            "attend": _exact_attend}[case["op"]](st)
