"""Trees of drafted tokens: kq_kv_append_tree, kq_attn_tree and kq_tree_accept against their definitions in 64 bits.

Bounds: those of tests/test_gpu_cache.py, where they are derived.  A tree only changes which position a token rotates by
and which products count, not how they are computed; where its masks say a chain, the results are a chain's within the same
bounds.
"""
import numpy as np
import pytest
import torch

from gguf_quant_weight_super_gb300 import kq
from tests.test_gpu_cache import BF16, F8, F32, Paged, _setup, attn_ref, check_attn, f64, rand_q  # noqa: F401

pytestmark = pytest.mark.gpu


def random_parents(T, r, nodes=None, wide=3):
    """Parents of a tree whose children follow their parents: -1 the root's, None for padding."""
    nodes = T if nodes is None else nodes
    return [None if t >= nodes else -1 if t == 0 else int(r.integers(max(0, (t - 1) // wide - 1), t)) for t in range(T)]


def masks_of(parents):
    m = []
    for t, p in enumerate(parents):
        m.append(0 if p is None else (1 << t) | (m[p] if p >= 0 else 0))
    return m


def chain(T):
    return [(2 << t) - 1 for t in range(T)]


def to_tensor(masks):
    a = np.array(masks, dtype=np.uint64).reshape(len(masks), -1)
    return torch.from_numpy(a.view(np.int64)).cuda()


def tree_tokens(masks, n):
    """Per token: (the drafted tokens that it sees, its position) or None for padding; n the sequence's length."""
    T = len(masks)
    there = {u for u in range(T) if n - T + u >= 0}
    out = []
    for t in range(T):
        see = [u for u in sorted(there) if masks[t] >> u & 1] if t in there else []
        out.append((see, max(0, n - T) + len(see) - 1) if see else None)
    return out


def tree_columns(masks, n, window):
    """Per token: the slots that it sees."""
    T, base = len(masks), n - len(masks)
    nodes = tree_tokens(masks, n)
    out = []
    for x in nodes:
        if x is None:
            out.append([])
            continue
        see, pos = x
        lo = max(0, pos - window + 1) if window else 0
        # a padding token's slot stands nowhere: position -1
        where = [nodes[u][1] if nodes[u] else -1 for u in see]
        out.append(list(range(lo, max(0, base))) + [base + u for u, w in zip(see, where) if not window or w > pos - window])
    return out


def tree_ref(P, masks, q, scale, cap, window):
    q = f64(q.float())
    B, T, Hq, D = q.shape
    out, sv, ds = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, T, Hq, 1))
    for b in range(B):
        k, v = P.dense(b)
        Hkv = k.shape[1]
        for t, cols in enumerate(tree_columns(masks[b], P.lens[b], window)):
            if not cols:
                continue
            for h in range(Hq):
                kk, vv = k[cols, h * Hkv // Hq], v[cols, h * Hkv // Hq]
                s = kk @ q[b, t, h] * scale
                ds[b, t, h] = (D + 8) * 2.0 ** -23 * abs(scale) * np.max(np.abs(kk) @ np.abs(q[b, t, h])) + cap * 2.0 ** -21
                if cap:
                    s = cap * np.tanh(s / cap)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, t, h], sv[b, t, h] = p @ vv, p @ np.abs(vv)
    return out, sv, ds


def check_tree(P, masks, q, scale=None, cap=0.0, window=0, skip=None):
    B, T, Hq, D = q.shape
    ws = kq.attn_tree_workspace(P.cache, B, T, Hq)
    tree = to_tensor(masks)
    out = torch.full((B, T, Hq, D), float("nan"), dtype=q.dtype, device="cuda")
    kq.attn_tree(P.cache, P.table, P.seq_lens, tree, q, ws, scale=scale, softcap=cap, window=window, out=out)
    torch.cuda.synchronize()
    ref, sv, ds = tree_ref(P, masks, q, D ** -0.5 if scale is None else scale, cap, window)
    n = max(1, max(P.lens))
    part, rnd = (2.0 ** -16, 2.0 ** -8) if q.dtype == BF16 else (2.0 ** -20, 2.0 ** -24)
    d = 2 * ds + 2.0 ** -20 + part + (n / 8 + 128) * 2.0 ** -23
    tol = d * sv * (1 + rnd) + rnd * np.abs(ref)
    err = np.abs(f64(out.float()) - ref)
    if skip is not None:
        err[skip], tol[skip] = 0.0, 0.0
    assert np.all(np.isfinite(err)) and np.all(err <= tol), float(np.nanmax(err / np.maximum(tol, 1e-300)))
    again = torch.empty_like(out)
    kq.attn_tree(P.cache, P.table, P.seq_lens, tree, q, ws, scale=scale, softcap=cap, window=window, out=again)
    torch.cuda.synchronize()
    assert torch.equal(again.isnan(), out.isnan()) and torch.equal(again.nan_to_num(), out.nan_to_num())
    return out


def trees(B, T, seed):
    r = np.random.default_rng(seed)
    return [masks_of(random_parents(T, r, nodes=T if b % 3 == 0 else max(1, T - int(r.integers(0, T))))) for b in range(B)]


# ---- attention

@pytest.mark.parametrize("q_dtype,dtype", [(BF16, BF16), (F32, BF16), (BF16, F8), (F32, F8)])
@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (128, 2, 4), (128, 1, 16), (256, 1, 2)])
@pytest.mark.parametrize("T", [1, 5, 16, 33])
def test_attn_tree(q_dtype, dtype, D, Hkv, G, T):
    lens = [T, 0, T + 1, T + 63, 300, max(1, T - 3)]
    P = Paged(lens, Hkv, D, 16, dtype, seed=T + D)
    check_tree(P, trees(len(lens), T, 5 * T + D), rand_q(len(lens), T, Hkv * G, D, q_dtype, 11 * T + G))


@pytest.mark.parametrize("q_dtype,G,D", [(BF16, 8, 128), (BF16, 3, 64), (F32, 2, 128)])
def test_attn_tree_of_64_nodes_split_over_the_device(q_dtype, G, D):
    lens = [5000, 64, 1024 + 37]
    P = Paged(lens, 1, D, 32, BF16, seed=3, layout="head")
    check_tree(P, trees(3, 64, 17), rand_q(3, 64, G, D, q_dtype, 5))


@pytest.mark.parametrize("q_dtype,dtype,T", [(BF16, BF16, 24), (F32, F8, 9), (BF16, BF16, 40)])
@pytest.mark.parametrize("window,cap", [(1, 0.0), (3, 30.0), (17, 0.0), (64, 50.0), (1000, 5.0)])
def test_attn_tree_window_and_cap(q_dtype, dtype, T, window, cap):
    """Windows that end inside the tree, at its root, in the context and before it."""
    lens = [T + 130, T, T + 1, max(1, T - 2)]
    P = Paged(lens, 2, 128, 16, dtype, seed=window)
    check_tree(P, trees(4, T, window), rand_q(4, T, 4, 128, q_dtype, window + T), cap=cap, window=window)


@pytest.mark.parametrize("q_dtype,dtype,G,T", [(BF16, BF16, 4, 7), (F32, F8, 2, 16), (BF16, BF16, 16, 16), (BF16, F8, 1, 1)])
@pytest.mark.parametrize("window", [0, 9])
def test_attn_tree_of_a_chain_is_attn_decode(q_dtype, dtype, G, T, window):
    lens = [700, T, 0, T + 64, 2000]
    P = Paged(lens, 2, 128, 16, dtype, seed=9)
    q = rand_q(5, T, 2 * G, 128, q_dtype, 2)
    # They may go to different kernels, and join a sequence's parts in another order: each is within the bound of the same
    # values, which are computed here from the lengths and there from the masks.
    one = check_attn(P, q, window=window)
    two = check_tree(P, [chain(T)] * 5, q, window=window)
    ref, ref2 = attn_ref(P, q, 128 ** -0.5, 0.0, window)[0], tree_ref(P, [chain(T)] * 5, q, 128 ** -0.5, 0.0, window)[0]
    assert np.array_equal(ref, ref2) and one.shape == two.shape


@pytest.mark.parametrize("q_dtype,dtype,G", [(BF16, BF16, 2), (BF16, BF16, 8), (F32, F8, 2)])
def test_attn_tree_values_that_are_not_finite_reach_only_who_sees_them(q_dtype, dtype, G):
    """NaN and infinities in a node, in padding's slots and behind the window; padding beside a context with NaN."""
    T = 12
    par = [-1, 0, 0, 1, 1, 2, 3, 3, None, None, None, None]
    masks = [masks_of(par)] * 3
    lens = [T + 200, T, T + 40]
    P = Paged(lens, 1, 128, 16, dtype, seed=1)
    for b, n in enumerate(lens):
        for u, x in ((3, float("nan")), (8, float("nan")), (11, float("inf") if dtype == BF16 else float("nan"))):
            j = n - T + u
            for pool in (P.k, P.v):
                pool[int(P.table[b, j // 16]), j % 16] = torch.tensor(x).to(dtype)
    j = 5  # of the third sequence's context: everybody but its padding sees it
    P.v[int(P.table[2, j // 16]), j % 16] = torch.tensor(float("nan")).to(dtype)
    sees3 = np.array([m >> 3 & 1 for m in masks[0]], dtype=bool)
    skip = np.zeros((3, T, G, 128), dtype=bool)
    skip[:, sees3] = True
    skip[2, :8] = True
    out = check_tree(P, masks, rand_q(3, T, G, 128, q_dtype, 4), skip=skip)
    assert out[:2].float()[:, torch.from_numpy(sees3)].isnan().all()
    assert torch.equal(out[:, 8:], torch.zeros_like(out[:, 8:]))


def test_attn_tree_sets_of_bits_that_are_no_ancestors():
    """Any bits, bits past T among them."""
    r = np.random.default_rng(8)
    T, lens = 20, [50, 20, 19, 300]
    masks = [[int(x) for x in r.integers(0, 2 ** 63, T)] for _ in lens]
    masks[0][3] = 0
    P = Paged(lens, 2, 64, 8, BF16, seed=2)
    check_tree(P, masks, rand_q(4, T, 8, 64, BF16, 3))


def padded_masks(r, T):
    """Any bits, few or many of them, a third of the tokens padding that others' bits name."""
    few = r.integers(0, 2, T)
    m = [int(r.integers(0, 2 ** 63) & (r.integers(0, 2 ** 63) if f else 2 ** 63 - 1)) & (1 << T) - 1 for f in few]
    return [0 if r.random() < 0.33 else x for x in m]


@pytest.mark.parametrize("q_dtype,dtype,D,G", [(BF16, BF16, 64, 1), (F32, F8, 128, 2), (BF16, BF16, 128, 4)])
@pytest.mark.parametrize("window", [1, 2, 3, 9, 16, 20, 21, 40, 57, 60, 61, 300, 319, 320, 1000])
def test_attn_tree_windows_and_bits_that_name_padding(q_dtype, dtype, D, G, window):
    """Padding stands at position -1: behind every window that ends after the sequence's start, however many bits a mask has.
    With four heads a group the call goes to the kernel of 128 rows."""
    r, T, lens = np.random.default_rng(window + G), 20, [60, 20, 19, 320]
    masks = [padded_masks(r, T) for _ in lens]
    masks[0][:6] = [1, 3, 0, 7, 0b10111, 0b101]
    masks[1][:3] = [0, 3, 7]
    masks[3][5] = (1 << T) - 1  # the newest position that there can be
    P = Paged(lens, 2, D, 16, dtype, seed=window)
    q = rand_q(4, T, 2 * G, D, q_dtype, window)
    check_tree(P, masks, q, window=window)
    P.table = P.table[:, :-1].contiguous()  # room for 320 positions, and no more
    check_tree(P, masks, q, window=window)


@pytest.mark.parametrize("q_dtype,dtype,D,G", [(F32, BF16, 128, 1), (BF16, F8, 64, 3), (BF16, BF16, 64, 4)])
@pytest.mark.parametrize("T,window", [(33, 5), (50, 17), (50, 60), (64, 33), (64, 90)])
def test_attn_tree_windows_and_padding_among_more_than_32_tokens(q_dtype, dtype, D, G, T, window):
    r, lens = np.random.default_rng(window + T), [T + 40, T, T - 1, 500]
    masks = [padded_masks(r, min(T, 62)) + [0, 5][:max(0, T - 62)] for _ in lens]
    masks[3][T - 1] = (1 << T) - 1
    P = Paged(lens, 2, D, 16, dtype, seed=window)
    check_tree(P, masks, rand_q(4, T, 2 * G, D, q_dtype, window), window=window)


# ---- append

def append_ref(P, masks, q, k, v, cs, rot, inter, wq, wk, off, eps):
    B, T = q.shape[:2]
    qs = np.zeros(q.shape)
    stored = {}
    half = rot // 2
    i = np.arange(half) * (2 if inter else 1)
    j = i + (1 if inter else half)

    def norm_turn(x, w, pos):
        if w is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (f64(w) + off)
        y = x.copy()
        c, s = cs[pos, :half], cs[pos, half:]
        y[:, i], y[:, j] = x[:, i] * c - x[:, j] * s, x[:, j] * c + x[:, i] * s
        return y, np.abs(x) + np.abs(np.concatenate([x[:, j], x[:, i]], 1)[:, np.argsort(np.concatenate([i, j]))] if rot == x.shape[1]
                                     else np.abs(x).max())
    mag = np.zeros(q.shape)
    for b in range(B):
        for t, x in enumerate(tree_tokens(masks[b], P.lens[b])):
            if x is None:
                continue
            pos, slot = x[1], P.lens[b] - T + t
            qs[b, t], mag[b, t] = norm_turn(f64(q[b, t].float()), wq, pos)
            kk, km = norm_turn(f64(k[b, t].float()), wk, pos)
            stored[int(P.table[b, slot // P.page]), slot % P.page] = (kk / P.k_scale, km / P.k_scale,
                                                                      f64(v[b, t].float()) / P.v_scale)
    return qs, mag, stored


def rounded(err, ref, mag, dtype):
    """Whether err is within the arithmetic's bound and one rounding to dtype (tests/test_gpu_cache.py)."""
    rnd = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F8: 2.0 ** -4}[dtype]
    least = 2.0 ** -10 if dtype == F8 else 0.0
    return np.all(err <= 2.0 ** -20 * mag * (1 + rnd) + np.maximum(rnd * np.abs(ref), least))


@pytest.mark.parametrize("T", [1, 6, 31, 64])
@pytest.mark.parametrize("x,out,dtype,D,rot,inter,norm", [
    (F32, BF16, BF16, 128, 128, False, True), (BF16, F32, F8, 256, 128, True, True), (F32, F32, F8, 64, 64, False, False),
    (BF16, BF16, BF16, 64, 32, True, False)])
def test_append_tree(T, x, out, dtype, D, rot, inter, norm):
    lens = [T + 33, 0, T, max(1, T - 2), T + 500]
    B, Hq, Hkv = len(lens), 6, 2
    P = Paged(lens, Hkv, D, 16, dtype, seed=T, fill="zero")
    masks = trees(B, T, T + 1)
    g = torch.Generator().manual_seed(T)
    fused = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g).to(x).cuda()
    q, k, v = fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv], fused[:, :, Hq + Hkv:]
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2)) if norm else (None, None)
    cs = kq.rope_table(T + 600, rot, base=500.0)
    r = kq.RopeNorm(cs, interleaved=inter, q_norm=wq, k_norm=wk, eps=1e-5, norm_offset=0.25)
    before = [p.clone() for p in (P.k, P.v)]
    got = kq.kv_append_tree(P.cache, P.table, P.seq_lens, to_tensor(masks), q, k, v, r, q_out_dtype=out)
    torch.cuda.synchronize()
    qs, mag, stored = append_ref(P, masks, q, k, v, f64(cs), rot, inter, wq, wk, 0.25, 1e-5)
    assert rounded(np.abs(f64(got.float()) - qs), qs, mag, out)
    for pool, was, e in ((P.k, before[0], 0), (P.v, before[1], 2)):
        now, was = f64(pool.float()), f64(was.float())
        for (page, slot), row in stored.items():
            assert rounded(np.abs(now[page, slot] - row[e]), row[e], row[1] if e == 0 else 0 * row[e], dtype)
            now[page, slot] = was[page, slot]
        assert np.array_equal(now, was, equal_nan=True)  # nothing else is written


def test_append_tree_of_a_chain_is_kv_append():
    T, lens = 9, [9, 100, 0, 4]
    outs = []
    for masks in (None, [chain(T)] * 4):
        P = Paged(lens, 2, 128, 16, BF16, seed=6, fill="zero")
        q, k, v = (rand_q(4, T, h, 128, F32, h) for h in (8, 2, 2))
        r = kq.RopeNorm(kq.rope_table(200, 128))
        got = (kq.kv_append(P.cache, P.table, P.seq_lens, q, k, v, r) if masks is None else
               kq.kv_append_tree(P.cache, P.table, P.seq_lens, to_tensor(masks), q, k, v, r))
        outs.append([got] + [p.nan_to_num(7.0) for p in (P.k, P.v)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# ---- the walk and the move

def walk(masks, n, tokens, ids):
    """(path, next, new length) by the definition."""
    T = len(masks)
    there = (1 << T) - 1 & ~((1 << max(0, T - n)) - 1)
    bits = [m & there if there >> t & 1 else 0 for t, m in enumerate(masks)]
    path = []
    if bits[0] & 1:
        path = [0]
        while True:
            cur = path[-1]
            kids = [u for u in range(cur + 1, T) if bits[u] == bits[cur] | 1 << u and tokens[u] == ids[cur]]
            if not kids:
                break
            path.append(kids[0])
    return path, (int(ids[path[-1]]) if path else -1), max(0, n - T) + len(path)


def accept_case(B, T, lens, seed, words=3):
    """Trees with few different words, so that walks go deep and siblings share words."""
    r = np.random.default_rng(seed)
    masks = [masks_of(random_parents(T, r, nodes=max(1, T - int(r.integers(0, 3))), wide=2)) for _ in range(B)]
    return masks, r.integers(0, words, (B, T)).astype(np.int32), r.integers(0, words, (B, T)).astype(np.int32)


@pytest.mark.parametrize("T", [1, 2, 13, 32, 33, 64])
@pytest.mark.parametrize("dtype,layout,layers,Hkv,D", [(BF16, "token", 3, 2, 128), (F8, "head", 1, 5, 64), (BF16, "token", 17, 1, 256)])
def test_accept(T, dtype, layout, layers, Hkv, D):
    lens = [T, T + 7, 0, max(0, T - 1), T + 200, T + 15]
    B = len(lens)
    Ps = [Paged(lens, Hkv, D, 8, dtype, seed=70, layout=layout) for _ in range(layers)]  # one table, other values
    g = torch.Generator().manual_seed(T)
    for P in Ps:
        for pool in (P.k, P.v):
            pool.copy_((torch.randn(pool.shape, generator=g) * 20).to(dtype))
    before = [[p.clone() for p in (P.k, P.v)] for P in Ps]
    masks, tokens, ids = accept_case(B, T, lens, T)
    path, count, nxt, new = kq.tree_accept(kq.CacheSet([P.cache for P in Ps]), Ps[0].table, Ps[0].seq_lens, to_tensor(masks),
                                           torch.from_numpy(tokens).cuda(), torch.from_numpy(ids).cuda())
    torch.cuda.synchronize()
    table = Ps[0].table.cpu().numpy()
    want = [[p.clone() for p in pools] for pools in before]
    for b in range(B):
        p, n, length = walk(masks[b], lens[b], tokens[b], ids[b])
        assert path[b].tolist() == p + [-1] * (T - len(p))
        assert (int(count[b]), int(nxt[b]), int(new[b])) == (len(p), n, length)
        base = max(0, lens[b] - T)
        for i, u in enumerate(p):
            for was, pools in zip(before, want):
                for x, y in zip(was, pools):
                    y[table[b, (base + i) // 8], (base + i) % 8] = x[table[b, (base + u) // 8], (base + u) % 8]
    for P, pools in zip(Ps, want):
        for x, y in zip((P.k, P.v), pools):
            assert torch.equal(x.float(), y.float())


def test_accept_without_caches_and_equal_siblings():
    masks = [masks_of([-1, 0, 0, 2, 1, 1])]
    tokens = torch.tensor([[9, 5, 5, 7, 7, 7]], dtype=torch.int32, device="cuda")
    ids = torch.tensor([[5, 7, 7, 1, 2, 3]], dtype=torch.int32, device="cuda")
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([6], dtype=torch.int32, device="cuda")
    path, count, nxt, new = kq.tree_accept(kq.CacheSet([]), table, lens, to_tensor(masks), tokens, ids)
    assert path.tolist() == [[0, 1, 4, -1, -1, -1]] and (int(count), int(nxt), int(new)) == (3, 2, 3)


def test_accept_pages_outside_the_pool_are_recorded():
    P = Paged([20], 1, 64, 8, BF16, seed=1)
    before = P.k.clone()
    P.table[0, 1] = 1000  # slots 8..15
    masks = [masks_of([-1, 0, 0, 2])]
    words = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    ids = torch.tensor([[2, 0, 3, 0]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([14], dtype=torch.int32, device="cuda")  # base 10: all in the bad page
    path, *_ = kq.tree_accept(kq.CacheSet([P.cache]), P.table, lens, to_tensor(masks), words, ids)
    torch.cuda.synchronize()
    assert path.tolist() == [[0, 2, 3, -1]]
    assert kq.kq_device_error(clear=True) == 4
    assert torch.equal(P.k.nan_to_num(3.0), before.nan_to_num(3.0))


# ---- together

def test_a_verified_tree_step_equals_the_chain_of_its_branch():
    """Append a tree, attend, accept, and attend again from the new length: the cache then is, bit for bit, the one that
    appending the branch as a chain gives; captured in a graph and replayed with other words, on another stream."""
    B, T, Hq, Hkv, D, ctx = 3, 11, 8, 2, 128, [40, 3, 130]
    masks, tokens, _ = accept_case(B, T, None, 12, words=50)
    parents = [[None if m == 0 else max([u for u in range(t) if m >> u & 1], default=-1) for t, m in enumerate(ms)] for ms in masks]

    def ids_for(seed):
        rr = np.random.default_rng(seed)
        ids = np.full((B, T), 999, dtype=np.int32)
        for b in range(B):
            cur = 0
            while kids := [u for u in range(T) if parents[b][u] == cur]:
                u = int(rr.choice(kids))
                ids[b, cur] = tokens[b, u]
                cur = u
        return ids
    lens = [c + T for c in ctx]
    P, Q = (Paged(lens, Hkv, D, 16, BF16, seed=21) for _ in range(2))
    q, k, v = (rand_q(B, T, h, D, BF16, h + 1) for h in (Hq, Hkv, Hkv))
    rope = kq.RopeNorm(kq.rope_table(200, D))
    tree, words, chosen = to_tensor(masks), torch.from_numpy(tokens).cuda(), torch.from_numpy(ids_for(0)).cuda()
    ws, caches = kq.attn_tree_workspace(P.cache, B, T, Hq), kq.CacheSet([P.cache])
    outs = {}

    def step():
        outs["q"] = kq.kv_append_tree(P.cache, P.table, P.seq_lens, tree, q, k, v, rope)
        outs["a"] = kq.attn_tree(P.cache, P.table, P.seq_lens, tree, outs["q"], ws)
        outs["path"], outs["count"], outs["next"], outs["new"] = kq.tree_accept(caches, P.table, P.seq_lens, tree, words, chosen)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for seed in (1, 2):
        chosen.copy_(torch.from_numpy(ids_for(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            path, n, length = walk(masks[b], lens[b], tokens[b], ids_for(seed)[b])
            assert outs["path"][b].tolist()[:len(path)] == path and len(path) > 1
            assert (int(outs["count"][b]), int(outs["next"][b]), int(outs["new"][b])) == (len(path), n, length)
            one = torch.tensor([length], dtype=torch.int32, device="cuda")
            pick = torch.tensor(path, device="cuda")
            qc = kq.kv_append(Q.cache, Q.table[b:b + 1], one, *(x[b:b + 1, pick].contiguous() for x in (q, k, v)), rope)
            assert torch.equal(qc[0], outs["q"][b, pick])
            for x, y in ((P.k, Q.k), (P.v, Q.v)):
                j = torch.arange(length, device="cuda")
                pages = P.table[b].long()[j // 16]
                assert torch.equal(x[pages, j % 16], y[Q.table[b].long()[j // 16], j % 16])
            # the chain's attention: its last token's sums are those of the branch's last node
            wc = kq.attn_workspace(Q.cache, 1, len(path), Hq)
            ac = kq.attn_decode(Q.cache, Q.table[b:b + 1], one, qc, wc)
            d = (ac[0].float() - outs["a"][b, pick].float()).abs()
            # both are within one bf16 rounding and 2^-15 of sum p|v| (below 4) of the same value
            assert bool((d <= 2 * 2.0 ** -8 * ac[0].float().abs() + 2.0 ** -12).all())


# ---- many items, shared workspaces, long pools, other streams

@pytest.mark.parametrize("q_dtype,dtype,G,T", [(BF16, BF16, 4, 3), (F32, F8, 1, 2), (BF16, BF16, 8, 24)])
def test_attn_tree_more_sequences_than_ranges_and_one_split(q_dtype, dtype, G, T):
    """Parts joined range by range: 330 short sequences beside two that many ranges share."""
    lens = [int(x) for x in np.random.default_rng(4).integers(0, 60, 332)]
    lens[100], lens[331] = 9000, 5003
    P = Paged(lens, 1, 128, 16, dtype, seed=9)
    check_tree(P, trees(332, T, 3), rand_q(332, T, G, 128, q_dtype, 6))


def test_attn_tree_and_attn_decode_share_a_workspace():
    """In turn, on one stream, what the largest call asked for: splits or none, wide and narrow, trees and chains."""
    P = Paged([3000, 5, 0, 64, 900, 17], 2, 128, 16, BF16, seed=5)
    shapes = [(7, 8, BF16), (1, 2, BF16), (24, 16, BF16), (3, 4, F32), (64, 8, BF16), (2, 16, BF16)]
    ws = torch.zeros(max(kq.attn_tree_workspace(P.cache, 6, t, h).numel() for t, h, _ in shapes), dtype=torch.uint8, device="cuda")
    for rep in range(2):
        for t, h, d in shapes:
            q, tree = rand_q(6, t, h, 128, d, t + h + rep), to_tensor(trees(6, t, t))
            # a workspace of its own gives the same bits
            one = kq.attn_tree(P.cache, P.table, P.seq_lens, tree, q, ws)
            own = kq.attn_tree(P.cache, P.table, P.seq_lens, tree, q, kq.attn_tree_workspace(P.cache, 6, t, h))
            assert torch.equal(one, own), (rep, t, h)
            if t <= 16:  # chains of more are refused
                two = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws)
                own = kq.attn_decode(P.cache, P.table, P.seq_lens, q, kq.attn_workspace(P.cache, 6, t, h))
                assert torch.equal(two, own), (rep, t, h)


@pytest.mark.parametrize("q_dtype,dtype,G", [(BF16, BF16, 8), (F32, F8, 2)])
def test_tree_ops_in_pages_past_2_to_the_32_bytes_and_elements(q_dtype, dtype, G):
    T, lens, page, D = 9, [9, 700, 33], 32, 128
    P = Paged(lens, 2, D, page, dtype, seed=3)
    n = P.k.shape[0]
    far = -(-(2 ** 32 + 4096) // (page * 2 * D))
    pools = []
    for x in (P.k, P.v):
        pool = torch.empty((far + n, page, 2, D), dtype=dtype, device="cuda")
        pool[:far].view(torch.uint8).fill_(0xff)  # NaN
        pool[far:] = x
        pools.append(pool)
    table = torch.where(P.table >= 0, P.table + far, P.table)
    big = kq.KVCache(*pools, P.k_scale, P.v_scale)
    q, k, v = (rand_q(3, T, h, D, q_dtype, h) for h in (2 * G, 2, 2))
    tree, rope, ws = to_tensor(trees(3, T, 5)), kq.RopeNorm(kq.rope_table(800, D)), kq.attn_tree_workspace(P.cache, 3, T, 2 * G)
    g = torch.Generator().manual_seed(5)
    words, ids = (torch.randint(0, 2, (3, T), generator=g).int().cuda() for _ in range(2))
    outs = []
    for cache, tab in ((P.cache, P.table), (big, table)):
        a = kq.kv_append_tree(cache, tab, P.seq_lens, tree, q, k, v, rope, q_out_dtype=q_dtype)
        o = kq.attn_tree(cache, tab, P.seq_lens, tree, a, ws)
        outs.append([a, o, *kq.tree_accept(kq.CacheSet([cache]), tab, P.seq_lens, tree, words, ids)])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    for pool, x in zip(pools, (P.k, P.v)):
        assert torch.equal(pool[far:].view(torch.uint8), x.view(torch.uint8))
        assert bool((pool[:far].view(torch.int64) == -1).all())


def test_attn_tree_rows_with_strides_on_another_stream():
    """Queries inside a fused projection; a stream that waits for nothing else."""
    P = Paged([900, 40, 0], 2, 128, 16, BF16, seed=2)
    for T, Hq in ((4, 4), (24, 16)):
        masks = trees(3, T, 1)
        fused = rand_q(3, T, Hq + 5, 128, BF16, 3)
        q = fused[:, :, 2:2 + Hq]
        want = check_tree(P, masks, q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = kq.attn_tree(P.cache, P.table, P.seq_lens, to_tensor(masks), q, kq.attn_tree_workspace(P.cache, 3, T, Hq),
                           stream=side)
        side.synchronize()
        assert torch.equal(got, want)
