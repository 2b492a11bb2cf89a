"""Forking, freeing, compacting and copying pages on the GPU, against sequential lists (tests/_kv4_ref.py).
Everything is a whole number and must match exactly."""
import numpy as np
import pytest

from tests import _kv4_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_201_gb300 as pa
    pa.load_library(build_if_missing=True)
    pa.paged_attn_last_error_word()
    return pa


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _full(n, fill=-7):
    import torch
    return torch.full(n if isinstance(n, tuple) else (n,), fill, dtype=torch.int32, device="cuda")


def _bits(pa, want):
    bits = pa.paged_attn_last_error_word()
    assert bool(bits & pa.ERRBIT_REFUSED) == want["refused"]
    assert bool(bits & pa.ERRBIT_PAGE_RANGE) == want["bad"]
    return bits & ~(pa.ERRBIT_REFUSED | pa.ERRBIT_PAGE_RANGE)


def _same(got, want):
    np.testing.assert_array_equal(got.cpu().numpy(), np.asarray(want, np.int32).reshape(got.shape))


def _state(seed, B, width, ps, empty=0.3, shared=0.3, spare=40):
    """Rows over shuffled pages, some empty, some with a prompt in common, and the stack of the others."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, width * ps + 1, B)
    lens[rng.uniform(size=B) < 0.2] = width * ps // 2 // ps * ps
    lens[rng.uniform(size=B) < empty] = 0
    need = -(-lens // ps)
    P = int(need.sum()) + spare
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((B, width), 0x7FFFFFFF, np.int32)
    table[np.arange(width)[None] < need[:, None]] = ids[:int(need.sum())]
    for b in np.nonzero(rng.uniform(size=B) < shared)[0]:
        o = int(rng.integers(0, B))
        n = min(lens[b], lens[o]) // ps
        table[b, :n] = table[o, :n]
    listed = table[np.arange(width)[None] < need[:, None]]
    shares = np.zeros(P, np.int64)
    u, n = np.unique(listed, return_counts=True)
    shares[u] = n - 1
    free = rng.permutation(np.setdiff1d(np.arange(P), u))
    stack = np.full(P, -9, np.int32)
    stack[:len(free)] = free
    return dict(table=table, lens=lens.astype(np.int32), shares=shares.astype(np.int32), stack=stack, count=len(free),
                ps=ps, P=P, B=B, rng=rng)


# ----------------------------------------------------------------------------- fork
def _fork(pa, s, parents, children, prefix=None, count=None, alias=False, P=None, stack=None):
    stack = s["stack"] if stack is None else stack
    count = s["count"] if count is None else count
    P = s["P"] if P is None else P
    want = R.fork(parents, children, prefix, s["table"], s["lens"], s["shares"][:P], stack, count, s["ps"], P)
    table, lens, shares, free, cnt = _t(s["table"]), _t(s["lens"]), _t(s["shares"][:P]), _t(stack), _t([count])
    lens_out = lens if alias else _full(s["B"])
    left = cnt if alias else _full(1)
    copies = _full((len(parents), 2))
    pa.paged_attn_fork(_t(parents), _t(children), table, lens, lens_out, shares, free, cnt, left, copies, s["ps"],
                       prefix_lens=None if prefix is None else _t(prefix))
    _same(table, want["table"])
    _same(lens_out, want["lens"])
    _same(shares, want["shares"])
    _same(copies, want["copies"])
    _same(left, [want["left"]])
    _same(free, stack)
    return want, _bits(pa, want)


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("ps", [16, 32, 64])
@pytest.mark.parametrize("B,width,n", [(2, 1, 1), (9, 5, 3), (70, 30, 20), (1300, 9, 300), (3000, 4, 1500),
                                       (40, 700, 15)])
def test_fork(pa, B, width, n, ps, alias):
    s = _state(B + ps, B, width, ps, empty=0.6, spare=n + 3)
    s["lens"][0], s["lens"][-1] = max(1, s["lens"][0]), 0
    s["table"][0, 0] = s["table"][0, 0] if s["table"][0, 0] < s["P"] else 0
    free_rows, live = np.nonzero(s["lens"] == 0)[0], np.nonzero(s["lens"])[0]
    children = s["rng"].permutation(free_rows)[:n]
    parents = s["rng"].choice(live, len(children))
    want, rest = _fork(pa, s, parents, children, alias=alias)
    assert not want["refused"] and rest == 0
    prefix = s["rng"].integers(0, width * ps + 20, len(children))
    want, rest = _fork(pa, s, parents, children, prefix, alias=alias)
    assert not want["refused"] and rest == 0


@pytest.mark.parametrize("count", [0, 1, 5, -3, 10**6])
def test_fork_refusals(pa, count):
    """Too few pages, rows outside the table, children that are not empty, named twice or their own parents,
    negative prefixes; idle requests; a parent that is another's child counts as empty."""
    s = _state(5, 30, 6, 16, empty=0.5)
    e, l = np.nonzero(s["lens"] == 0)[0], np.nonzero(s["lens"])[0]
    parents = [l[0], -1, l[1], l[0], 30, -2, l[2], l[2], e[3], l[3], l[1], l[4], l[0], e[0]]
    children = [e[0], e[9], e[1], e[0], e[2], e[2], l[1], l[2], e[4], e[5], -1, e[6], e[7], e[8]]
    prefix = [10**6, 4, 3, 8, 8, 8, 8, 8, 8, -1, 5, 33, 16, 7]
    want, _ = _fork(pa, s, parents, children, prefix, count=count)
    assert want["refused"]
    want, _ = _fork(pa, s, parents, children, count=count, alias=True)
    assert want["refused"]


def test_fork_bad_pages(pa):
    """Ids outside the pool in a parent's row and in the stack; lengths past the row."""
    s = _state(6, 8, 4, 16, empty=0)
    s["lens"][4:] = 0
    s["lens"][:4] = [64, 40, 37, 1000]
    s["table"][:4] = np.arange(16).reshape(4, 4)
    s["table"][0, 1], s["table"][1, 2] = -1, 10**6
    stack = s["stack"].copy()
    stack[s["count"] - 2] = s["P"]
    want, rest = _fork(pa, s, [0, 1, 2, 3], [4, 5, 6, 7], stack=stack)
    assert want["bad"] and rest == pa.ERRBIT_SEQ_CLIPPED


def test_fork_nothing(pa):
    s = _state(7, 5, 4, 16)
    _fork(pa, s, [], [])
    _fork(pa, s, [-1, -1], [0, 99])


# ----------------------------------------------------------------------------- free
def _free(pa, s, rows, alias=False, count=None, stack=None, table=None):
    stack = s["stack"] if stack is None else stack
    count = s["count"] if count is None else count
    table = s["table"] if table is None else table
    want = R.free(list(rows), table, s["lens"], s["shares"], stack, count, s["ps"], s["P"])
    lens, shares, free, cnt = _t(s["lens"]), _t(s["shares"]), _t(stack), _t([count])
    lens_out, left = (lens, cnt) if alias else (_full(s["B"]), _full(1))
    pa.paged_attn_free(_t(rows), _t(table), lens, lens_out, shares, free, cnt, left, s["ps"])
    _same(lens_out, want["lens"])
    _same(shares, want["shares"])
    _same(free, want["stack"])
    _same(left, [want["left"]])
    return want, _bits(pa, want)


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("shared", [0.0, 0.7])
@pytest.mark.parametrize("B,width,n", [(1, 1, 1), (9, 5, 4), (70, 30, 70), (1300, 20, 1000), (3000, 4, 2500),
                                       (40, 700, 40), (200, 600, 190)])
def test_free(pa, B, width, n, shared, alias):
    for ps in (16, 64):
        s = _state(B + width + ps, B, width, ps, empty=0.1, shared=shared)
        want, rest = _free(pa, s, s["rng"].permutation(B)[:n], alias)
        assert not want["refused"] and not want["bad"] and rest == 0


def test_free_all_copies_of_a_prompt(pa):
    """Thirty rows with one list of pages, given up at once, in part and one by one."""
    s = _state(1, 30, 50, 16, empty=0)
    s["lens"][:] = 50 * 16
    s["table"][:] = s["rng"].permutation(s["P"])[:50]
    s["shares"][:] = 0
    s["shares"][s["table"][0]] = 29
    s["stack"][:] = -9
    s["count"] = 0
    want, _ = _free(pa, s, s["rng"].permutation(30))
    assert want["left"] == 50
    want, _ = _free(pa, s, [3, 7, 29])
    assert want["left"] == 0


def test_free_refusals(pa):
    """Rows named twice, idle ones, rows outside the table, a stack without room, bad counts, ids outside the
    pool, negative lengths and such past the row."""
    s = _state(2, 12, 6, 16, empty=0)
    _free(pa, s, [3, 3, 5, -1, 3, 5])
    want, _ = _free(pa, s, [3, 12, -2, 4])
    assert want["refused"]
    want, _ = _free(pa, s, [1, 2, 3], stack=s["stack"][:s["count"] + 4])
    assert want["refused"] and want["left"] == s["count"] + 4
    for count in (-1, 10**6):
        want, _ = _free(pa, s, [1, 2], count=count)
        assert want["refused"]
    table = s["table"].copy()
    table[4, 0], table[5, 0] = -1, s["P"]
    want, _ = _free(pa, s, [4, 5, 6], table=table)
    assert want["bad"]
    s["lens"][7], s["lens"][8] = -40, 5000
    s["table"][8] = s["stack"][:6]  # six pages that nobody lists
    want, rest = _free(pa, s, [7, 8, 9])
    assert rest == pa.ERRBIT_SEQ_CLIPPED
    _free(pa, s, [])


def test_free_restores_the_stack(pa):
    """What step_tables and fork took, given back in the same order, lies where it was."""
    import torch
    B, W, ps, P = 40, 12, 16, 600
    rng = np.random.default_rng(3)
    table, lens, shares = _full((B, W), -1), _full(B, 0), _full(P, 0)
    free, count = _t(rng.permutation(P)), _t([P])
    before = free.clone()
    new = rng.integers(1, W * ps, B)
    new[20:] = 0
    pa.paged_attn_step_tables(lens, _t(new), free, count, table, lens, _full(B), _full(B + 1), _full(int(new.sum())),
                              count, ps, P)
    copies = _full((20, 2))
    pa.paged_attn_fork(_t(np.arange(20)), _t(np.arange(20, 40)), table, lens, lens, shares, free, count, count, copies,
                       ps)
    pa.free_sequences(_t(np.arange(20, 40)), table, lens, shares, free, count, ps)
    pa.free_sequences(_t(np.arange(20)), table, lens, shares, free, count, ps)
    assert torch.equal(free, before) and int(count) == P and not shares.any() and not lens.any()
    assert pa.paged_attn_last_error_word() == 0


# ----------------------------------------------------------------------------- compact
def _compact(pa, s, stack=None, count=None, table=None):
    stack = s["stack"] if stack is None else stack
    count = s["count"] if count is None else count
    table = s["table"] if table is None else table
    want = R.compact(table, s["lens"], s["shares"], stack, count, s["ps"], s["P"])
    tab, shares, free, cnt = _t(table), _t(s["shares"]), _t(stack), _t([count])
    moves, n_moves, page_map = _full((s["P"] // 2, 2)), _full(1), _full(s["P"])
    pa.paged_attn_compact(tab, _t(s["lens"]), shares, free, cnt, moves, n_moves, page_map, s["ps"])
    _same(n_moves, [len(want["moves"])])
    all_moves = np.full((s["P"] // 2, 2), -7)
    if want["moves"]:
        all_moves[:len(want["moves"])] = want["moves"]
    _same(moves, all_moves)
    _same(tab, want["table"])
    _same(shares, want["shares"])
    _same(page_map, want["page_map"])
    _same(free, want["stack"])
    _same(cnt, [want["left"]])
    return want, _bits(pa, want)


@pytest.mark.parametrize("B,width,spare", [(1, 1, 1), (1, 3, 0), (5, 4, 7), (40, 30, 400), (300, 20, 3000), (20, 9, 9000),
                                           (2000, 9, 5000)])
def test_compact(pa, B, width, spare):
    for ps in (16, 32):
        s = _state(B + spare + ps, B, width, ps, empty=0.4, spare=spare)
        want, rest = _compact(pa, s)
        assert not want["refused"] and not want["bad"] and rest == 0


def test_compact_reserved_pages(pa):
    """Pages that are neither listed nor free stay, and stay unused; nothing free, nothing used."""
    s = _state(4, 30, 10, 16, empty=0.3, spare=200)
    _compact(pa, s, count=s["count"] // 2)
    _compact(pa, s, count=0)
    s["lens"][:] = 0
    want, _ = _compact(pa, s)
    assert not want["moves"]


def test_compact_odd_states(pa):
    """A free page that is listed, one that is free twice, ids outside the pool, bad counts."""
    s = _state(5, 12, 6, 16, empty=0, spare=60)
    stack = s["stack"].copy()
    stack[3] = s["table"][0, 0]
    stack[4] = stack[5]
    stack[6], stack[7] = -1, s["P"]
    table = s["table"].copy()
    table[1, 0], table[2, 0] = -1, 10**6
    want, _ = _compact(pa, s, stack=stack, table=table)
    assert want["refused"] and want["bad"]
    for count in (-1, 10**6):
        want, _ = _compact(pa, s, count=count)
        assert want["refused"]


def test_compact_largest_pools(pa):
    """Long runs of pages for every warp, and a count that is no multiple of anything."""
    s = _state(6, 64, 500, 16, empty=0.2, spare=200001)
    want, _ = _compact(pa, s)
    assert len(want["moves"]) > 10000


# ----------------------------------------------------------------------------- copies
def test_copy_pages(pa):
    """Pools of every kind at once; idle pairs, ids outside the pool, a count on the device."""
    import torch
    P = 50
    shapes = [((P, 3, 9 * 16 * 8), torch.uint8), ((P, 16, 2, 64), torch.bfloat16), ((P, 3), torch.float32),
              ((P, 1), torch.int32), ((P, 2, 2, 64), torch.int8), ((P, 70001), torch.int32), ((P, 32, 5, 256), torch.float32)]
    pools = [torch.randint(0, 256, s, device="cuda").to(d) for s, d in shapes]
    odd = torch.randint(0, 99, (P * 4 + 1,), device="cuda", dtype=torch.int32)[1:].view(P, 4)  # 4-byte aligned only
    pools.append(odd)
    pairs = [[3, 40], [-1, 5], [7, -1], [7, 41], [49, 0], [8, 8], [50, 1], [2, 2**31 - 1], [-5, 9], [20, 21]]
    for n in (None, 0, 5, 10, 100, -3):
        want = [p.clone() for p in pools]
        use = len(pairs) if n is None else max(0, min(n, len(pairs)))
        for a, b in pairs[:use]:
            if 0 <= a < P and 0 <= b < P:
                for w in want:
                    w[b] = w[a]
        pa.paged_attn_copy_pages(pools, _t(pairs), None if n is None else _t([n]))
        assert all(torch.equal(p, w) for p, w in zip(pools, want))
        assert pa.paged_attn_last_error_word() == (pa.ERRBIT_PAGE_RANGE if use > 6 else 0)
    pa.paged_attn_copy_pages(pools, _full((0, 2)))


# ----------------------------------------------------------------------------- together
def test_a_life_of_sequences(pa):
    """Prompts, forks, steps, ends and a compaction over a 4-bit pool and a 16-bit one with envelopes: after every step
    each sequence's attention is that of its own tokens, whoever shares them."""
    import torch
    torch.manual_seed(2)
    B, W, ps, Hkv, G, D, P = 12, 24, 16, 2, 4, 128, 400
    kv = pa.kv4_pool(P, ps, Hkv, D)
    kd, vd = (torch.zeros((P, ps, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    env, env_scale = pa.page_envelopes(kd)
    pools = [kv, kd, vd, env, env_scale]
    table, lens, shares = _full((B, W), -1), _full(B, 0), _full(P, 0)
    free, count = _t(torch.randperm(P).numpy()), _t([P])
    told = [None] * B  # every sequence's K and V rows, [2, tokens, Hkv, D]

    def step(new):
        nonlocal lens, count
        T = sum(new)
        rows = torch.randn((2, T, Hkv, D), device="cuda").bfloat16()
        lens, q_offset, q_start, slots, count = pa.step_tables(lens, _t(new), free, count, table, T, ps, P)
        pa.paged_attn_append_kv4(rows[0], rows[1], slots, kv)
        pa.paged_attn_append(rows[0], rows[1], slots, kd, vd, env, env_scale)
        at = 0
        for b, n in enumerate(new):
            if n:
                told[b] = rows[:, at:at + n] if told[b] is None else torch.cat([told[b], rows[:, at:at + n]], 1)
            at += n
        check()

    def check():
        q = torch.randn((B, 1, Hkv * G, D), device="cuda").bfloat16()
        out = pa.attention_kv4(q, kv, table, lens)
        dense = pa.attention(q, kd, vd, table, lens)
        for b in range(B):
            n = 0 if told[b] is None else told[b].shape[1]
            assert int(lens[b]) == n
            if n == 0:
                assert not out[b].any()
                continue
            pool = np.zeros((-(-n // ps), Hkv, 9 * ps * D // 8), np.uint8)
            x = told[b].double().cpu().numpy()
            R.write(pool, np.arange(n), x[0], x[1], ps)
            want, _, _, room, mass = R.attention(q[b].double().cpu().numpy(), pool, ps, np.arange(len(pool))[None], [n],
                                                 [0, 1], True, None, D ** -0.5)
            bar = 2.0 ** -8 * np.abs(want) + room + 2.0 ** -11 * mass  # as in test_kv4_gpu.py
            assert (np.abs(out[b].double().cpu().numpy() - want) <= bar).all()
            s = torch.einsum("hgd,nhd->hgn", q[b, 0].view(Hkv, G, D).double(), told[b][0].double()) * D ** -0.5
            want = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), told[b][1].double()).reshape(Hkv * G, D)
            assert ((dense[b, 0].double() - want).abs() <= 2e-3 + 2.0 ** -8 * want.abs()).all()

    step([70, 33, 48, 5] + [0] * 8)
    pa.fork_sequences(_t([0, 0, 2, 1, 3]), _t([4, 5, 6, 7, 8]), table, lens, shares, free, count, pools, ps)
    for a, b in ((0, 4), (0, 5), (2, 6), (1, 7), (3, 8)):
        told[b] = told[a].clone()
    check()
    step([1, 1, 1, 1, 1, 20, 1, 1, 40, 0, 0, 0])
    pa.free_sequences(_t([0, 5, 3]), table, lens, shares, free, count, ps)
    for b in (0, 5, 3):
        told[b] = None
    check()
    pa.fork_sequences(_t([8, 4]), _t([0, 9]), table, lens, shares, free, count, pools, ps, prefix_lens=_t([35, 48]))
    told[0], told[9] = told[8][:, :35].clone(), told[4][:, :48].clone()
    check()
    page_map, n_moves = pa.compact_pages(table, lens, shares, free, count, pools, ps)
    assert int(n_moves) > 0
    used = P - int(count)
    assert sorted(free[:int(count)].tolist()) == list(range(used, P))
    check()
    step([9, 1, 1, 0, 1, 3, 1, 1, 1, 1, 17, 0])
    pa.free_sequences(_t(np.arange(B)), table, lens, shares, free, count, ps)
    assert int(count) == P and not shares.any() and sorted(free.tolist()) == list(range(P))
    assert pa.paged_attn_last_error_word() == 0


def test_captured(pa):
    """A fork, its copies and a free in one graph, replayed: the state comes back every time."""
    import torch
    P, ps, W = 64, 16, 8
    pool = torch.randint(0, 256, (P, 1, 9 * ps * 8), dtype=torch.uint8, device="cuda")
    table = _full((4, W), -1)
    table[0, :3] = _t([5, 6, 7])
    lens, shares, count = _t([40, 0, 0, 0]), _full(P, 0), _t([P - 3])
    free = _t([p for p in range(P) if p not in (5, 6, 7)])
    before = free.clone()
    parents, children = _t([0, 0]), _t([2, 3])
    pa.paged_attn_last_error_word()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies = pa.fork_sequences(parents, children, table, lens, shares, free, count, [pool], ps)
        shown = torch.stack([lens, shares[5:9].clone()])
        pa.free_sequences(children, table, lens, shares, free, count, ps)
    for _ in range(3):
        pool[7] = torch.randint(0, 256, pool[7].shape, dtype=torch.uint8, device="cuda")
        graph.replay()
        torch.cuda.synchronize()
        assert shown.tolist() == [[40, 0, 40, 40], [2, 2, 0, 0]]
        assert copies.tolist() == [[7, 63], [7, 62]] and torch.equal(pool[63], pool[7])
        assert lens.tolist() == [40, 0, 0, 0] and not shares.any() and torch.equal(free, before) and int(count) == P - 3
    assert pa.paged_attn_last_error_word() == 0
