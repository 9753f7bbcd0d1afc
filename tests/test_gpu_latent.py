"""Latent caches: kq_latent_append, kq_latent_attn and kq_latent_accept against their definitions in 64 bits.

Bounds (derived, per element).
append.  As kq_kv_append's (tests/test_gpu_cache.py); the norm's sum has at most 512 terms, 16 a lane and then a tree, so
the same 2^-20 holds.
attention.  A score is a (latent + rope)-term fp32 sum of exact products, in two halves (the tensor cores may truncate:
2^-23 a step): |ds| <= (W + 8) 2^-23 scale sum|q c|, and the weights' relative error is 2 max|ds| + 2^-20 (exp).  They
enter the second product as bf16, 2^-8, and the sums over n positions add at most (n/8 + 128) 2^-23.  All of it
multiplies sum_j p_j |c_j|; then one rounding of the result, 2^-8.
Rounding errors of the weights are independent, so over the latent's many dims the error's mean square is far below that
bound's: a weight's rounding error is at most 2^-8 and 2^-8 / sqrt(3) in the mean square at most, so the sum's is
2^-8 / sqrt(3) sqrt(sum p^2 c^2); twice that and the other terms as they are bound a row's root mean square error.
"""
import numpy as np
import pytest
import torch

from gguf_quant_weight_super_gb300 import kq, synth
from tests.gpu_util import TOL
from tests.test_gpu_cache import BF16, F8, F32, _setup, f64  # noqa: F401
from tests.test_gpu_tree import chain, masks_of, rounded, to_tensor, tree_columns, tree_tokens, trees, walk

pytestmark = pytest.mark.gpu


class Latent:
    """A latent cache whose pages lie in any order; slots no sequence has hold NaN."""

    def __init__(self, lens, C, R, page, dtype, seed, pad=0, fill="random"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.C, self.R = list(lens), page, C, R
        used = [-(-max(0, n) // page) for n in lens]
        n_pages = sum(used) + 2
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), max(1, max(used, default=1)) + 1), -5, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = perm[at:at + u]
            at += u
        x = torch.randn((n_pages, page, C + R), generator=g) if fill == "random" else torch.zeros((n_pages, page, C + R))
        seen = torch.zeros((n_pages, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(used[b]):
                seen[table[b, i], :min(page, n - i * page)] = True
        self.scale = 0.25 if dtype == F8 else 1.0
        x = torch.where(seen[:, :, None], x / self.scale, float("nan")).to(dtype).cuda()
        mem = torch.zeros((n_pages, page, C + R + pad), device="cuda").to(dtype)
        self.c = mem[:, :, :C + R]
        self.c.copy_(x)
        self.table = table.cuda()
        self.cache = kq.LatentCache(self.c, C, self.scale)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()

    def dense(self, b):
        j = np.arange(max(0, self.lens[b]))
        return f64(self.c.float())[self.table[b].cpu().numpy()[j // self.page], j % self.page] * self.scale


def columns(masks, n, T):
    if masks is not None:
        return tree_columns(masks, n, 0)
    return [list(range(max(0, n - T + t + 1))) for t in range(T)]


def latent_q(B, T, H, W, seed, mul=1.4):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, T, H, W), generator=g) * mul).to(BF16).cuda()


def check_latent(P, q, masks=None, scale=None, skip=None, stream=None, ws=None):
    B, T, H, W = q.shape
    scale = (128 + P.R) ** -0.5 if scale is None else scale
    ws = kq.latent_attn_workspace(P.cache, B, T, H) if ws is None else ws
    tree = None if masks is None else to_tensor(masks)
    out = torch.full((B, T, H, P.C), float("nan"), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, scale, tree=tree, out=out, stream=stream)
    torch.cuda.synchronize()
    got, qn = f64(out.float()), f64(q.float())
    for b in range(B):
        c = P.dense(b)
        for t, cols in enumerate(columns(None if masks is None else masks[b], P.lens[b], T)):
            if skip is not None and skip[b][t]:
                continue
            if not cols:
                assert np.array_equal(got[b, t], np.zeros((H, P.C))), (b, t)
                continue
            k = c[cols]
            s = qn[b, t] @ k.T * scale
            ds = (W + 8) * 2.0 ** -23 * abs(scale) * np.max(np.abs(qn[b, t]) @ np.abs(k).T, axis=1)[:, None]
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            v = k[:, :P.C]
            ref, sv, sq = p @ v, p @ np.abs(v), np.sqrt((p * p) @ (v * v))
            rest = 2 * ds + 2.0 ** -20 + (len(cols) / 8 + 128) * 2.0 ** -23
            err = np.abs(got[b, t] - ref)
            tol = (rest + 2.0 ** -8) * sv * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
            assert np.all(np.isfinite(err)) and np.all(err <= tol), (b, t, float(np.nanmax(err / tol)))
            # and in the root mean square over a row: rounding of weights and of the result
            rms = np.sqrt((err ** 2).mean(1))
            most = np.sqrt((((2 * 2.0 ** -8 / 3 ** 0.5) * sq + rest * sv + 2.0 ** -8 * np.abs(ref)) ** 2).mean(1))
            assert np.all(rms <= most), (b, t, float((rms / most).max()))
    again = torch.empty_like(out)
    kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, scale, tree=tree, out=again)
    torch.cuda.synchronize()
    assert torch.equal(again.nan_to_num(), out.nan_to_num()) and torch.equal(again.isnan(), out.isnan())
    return out


# ---- attention

@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("C,R", [(512, 64), (256, 64), (512, 32), (256, 32)])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (1, 128), (3, 20), (2, 80)])
def test_latent_attn(dtype, C, R, T, H):
    lens = [1, 0, T, 63, 64, 65, 700]
    P = Latent(lens, C, R, 16, dtype, seed=C + R + H)
    check_latent(P, latent_q(len(lens), T, H, C + R, T + H))


@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("page", [1, 8, 64, 256])
def test_latent_attn_pages_strides_and_splits(dtype, page):
    """Pages that end inside tiles, padded rows, sequences split over the whole device beside ones of a few positions."""
    lens = [9001, 3, 0, 2049]
    P = Latent(lens, 512, 64, page, dtype, seed=page, pad=32)
    check_latent(P, latent_q(4, 1, 16, 576, page))


@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("T,H,L", [(1, 16, 70001), (9, 16, 30011), (1, 40, 50000), (2, 56, 40000), (1, 128, 40003), (3, 100, 20011)])
def test_latent_attn_long_segments(dtype, T, H, L):
    """Every range a dozen tiles, with all rows of a tile, some, few."""
    P = Latent([L, 77], 512, 64, 64, dtype, seed=T + H)
    check_latent(P, latent_q(2, T, H, 576, T + H))


def test_latent_attn_many_sequences_and_rows():
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 400, 70)]
    P = Latent(lens, 512, 64, 32, BF16, seed=5)
    check_latent(P, latent_q(70, 1, 24, 576, 6))
    P = Latent([300, 77, 16], 512, 64, 32, BF16, seed=6)
    check_latent(P, latent_q(3, 16, 40, 576, 7))  # 640 rows a sequence


@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("T,H", [(1, 16), (9, 16), (33, 4), (64, 3), (7, 128)])
def test_latent_attn_tree(dtype, T, H):
    lens = [T, 0, T + 1, T + 300, max(1, T - 3)]
    P = Latent(lens, 512, 64, 16, dtype, seed=T)
    check_latent(P, latent_q(5, T, H, 576, T + H), trees(5, T, T))


def test_latent_attn_chain_as_a_tree_gives_the_same():
    T, lens = 6, [6, 500, 0, 4, 2000]
    P = Latent(lens, 512, 64, 16, BF16, seed=2)
    q, ws = latent_q(5, T, 16, 576, 3), kq.latent_attn_workspace(P.cache, 5, T, 16)
    one = kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, 0.07)
    two = kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, 0.07, tree=to_tensor([chain(T)] * 5))
    assert torch.equal(one, two)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 30.0])
def test_latent_attn_scales(scale):
    """No scale: the mean.  A negative one: the order turns around.  Large ones: one position takes all."""
    P = Latent([100, 1, 1500], 512, 64, 16, BF16, seed=8)
    check_latent(P, latent_q(3, 2, 8, 576, 4), scale=scale)


@pytest.mark.parametrize("up", [False, True])
def test_latent_attn_scores_that_grow_along_the_sequence(up):
    """Each tile's largest score above (below) the last one's by many powers of two."""
    P = Latent([2000], 512, 64, 16, BF16, seed=8)
    g = torch.linspace(0.0, 3.0, 2000, device="cuda") if up else torch.linspace(3.0, 0.0, 2000, device="cuda")
    j = torch.arange(2000, device="cuda")
    P.c[P.table[0].long()[j // 16], j % 16, 3] = (g * 20).to(BF16)
    q = latent_q(1, 1, 16, 576, 4, mul=0.3)
    q[..., 3] = 20.0
    check_latent(P, q)


@pytest.mark.parametrize("dtype", [BF16, F8])
def test_latent_attn_vectors_that_are_not_finite_reach_only_who_sees_them(dtype):
    T = 10
    par = [-1, 0, 0, 1, 1, 2, 3, None, None, None]
    masks, lens = [masks_of(par)] * 3, [T + 150, T, T + 60]
    P = Latent(lens, 512, 64, 16, dtype, seed=1)
    bad = torch.tensor(float("nan")).to(dtype)
    for b, n in enumerate(lens):
        for u, d in ((3, 7), (7, 300), (9, 570)):  # in either half of the latent, in the rope part
            j = n - T + u
            P.c[int(P.table[b, j // 16]), j % 16, d] = bad
    P.c[int(P.table[2, 0]), 5, 511] = bad  # in the third sequence's context: everybody but its padding sees it
    skip = [[bool(m >> 3 & 1) or (b == 2 and m != 0) for m in masks[0]] for b in range(3)]
    out = check_latent(P, latent_q(3, T, 16, 576, 4), masks, skip=skip)
    assert torch.equal(out[:, 7:], torch.zeros_like(out[:, 7:]))
    # a chain: the newest token's vector reaches the newest token only
    P = Latent([200, 3], 512, 64, 16, BF16, seed=1)
    P.c[int(P.table[0, 199 // 16]), 199 % 16, 40] = float("inf")
    check_latent(P, latent_q(2, 3, 16, 576, 4), skip=[[False, False, True], [False] * 3])


def test_latent_attn_a_query_that_is_not_finite_reaches_no_other_row():
    P = Latent([500, 40], 512, 64, 16, BF16, seed=1)
    q = latent_q(2, 2, 16, 576, 4)
    clean = check_latent(P, q)
    q[0, 1, 5, 17] = float("nan")
    q[1, 0, 2, 570] = float("inf")
    ws = kq.latent_attn_workspace(P.cache, 2, 2, 16)
    out = kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, (128 + 64) ** -0.5)
    keep = torch.ones((2, 2, 16), dtype=torch.bool, device="cuda")
    keep[0, 1, 5] = keep[1, 0, 2] = False
    assert torch.equal(out[keep], clean[keep])


def test_latent_attn_lengths_and_pages_outside_are_recorded():
    P = Latent([100], 512, 64, 16, BF16, seed=1)
    q, ws = latent_q(1, 1, 4, 576, 4), kq.latent_attn_workspace(P.cache, 1, 1, 4)
    P.seq_lens.fill_(10 ** 6)
    P.table[P.table < 0] = 0
    kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, 0.1)
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 4
    P.seq_lens.fill_(100)
    P.table[0, 2] = 77
    kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, 0.1)
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 4
    P.table[0, 2] = -1
    kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, 0.1)
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 4
    P = Latent([100], 512, 64, 16, BF16, seed=1)
    check_latent(P, q, ws=ws)  # the workspace is as it was


# ---- append

@pytest.mark.parametrize("x,dtype", [(F32, BF16), (BF16, BF16), (F32, F8), (BF16, F8)])
@pytest.mark.parametrize("C,R,H,inter,norm", [(512, 64, 16, True, True), (256, 32, 5, False, True), (512, 32, 1, False, False),
                                              (256, 64, 7, True, False)])
@pytest.mark.parametrize("T,tree", [(1, False), (5, False), (130, False), (7, True), (64, True)])
def test_latent_append(x, dtype, C, R, H, inter, norm, T, tree):
    lens = [T, T + 40, 0, max(1, T - 3)]
    B, W = len(lens), C + R
    P = Latent(lens, C, R, 16, dtype, seed=T, pad=16, fill="zero")
    masks = trees(B, T, T) if tree else None
    g = torch.Generator().manual_seed(T + C)
    c = torch.randn((B, T, W + 16), generator=g).to(x).cuda()[:, :, :W]
    ql = torch.randn((B, T, H, C), generator=g).to(x).cuda()
    qr = torch.randn((B, T, H, 48 + R), generator=g).to(x).cuda()[..., 48:]
    w = (1 + 0.2 * torch.randn(C, generator=g)).cuda() if norm else None
    cs = kq.rope_table(T + 100, R, base=300.0)
    rope = kq.RopeNorm(cs, interleaved=inter, k_norm=w, eps=1e-5, norm_offset=0.5)
    before = P.c.clone()
    got = kq.latent_append(P.cache, P.table, P.seq_lens, ql, qr, c, rope, tree=None if masks is None else to_tensor(masks))
    torch.cuda.synchronize()
    tab, half = f64(cs), R // 2
    i = np.arange(half) * (2 if inter else 1)
    j = i + (1 if inter else half)

    def turn(v, pos):
        y, m = v.copy(), np.abs(v)
        y[..., i], y[..., j] = (v[..., i] * tab[pos, :half] - v[..., j] * tab[pos, half:],
                                v[..., j] * tab[pos, :half] + v[..., i] * tab[pos, half:])
        m[..., i] = m[..., j] = np.abs(v[..., i]) + np.abs(v[..., j])
        return y, m
    now, was = f64(P.c.float()), f64(before.float())
    for b, n in enumerate(lens):
        for t in range(T):
            pos = n - T + t
            if tree:
                node = tree_tokens(masks[b], n)[t]
                pos = -1 if node is None else node[1]
            if pos < 0:
                assert torch.equal(got[b, t], torch.zeros_like(got[b, t]))
                continue
            a, r = f64(ql[b, t].float()), turn(f64(qr[b, t].float()), pos)
            ref, mag = np.concatenate([a, r[0]], 1), np.concatenate([np.abs(a), r[1]], 1)
            assert rounded(np.abs(f64(got[b, t].float()) - ref), ref, mag, BF16)
            row = f64(c[b, t].float())
            v = row[:C]
            if norm:
                v = v / np.sqrt((v * v).mean() + 1e-5) * (f64(w) + 0.5)
            r = turn(row[C:], pos)
            ref, mag = np.concatenate([v, r[0]]) / P.scale, np.concatenate([np.abs(v), r[1]]) / P.scale
            at = int(P.table[b, (n - T + t) // 16]), (n - T + t) % 16
            assert rounded(np.abs(now[at] - ref), ref, mag, dtype)
            now[at] = was[at]
    assert np.array_equal(now, was, equal_nan=True)  # nothing else is written


def test_latent_append_positions_outside_the_table_are_recorded():
    P = Latent([30], 512, 64, 16, BF16, seed=1)
    before = P.c.clone()
    rope = kq.RopeNorm(kq.rope_table(20, 64))
    x = torch.ones((1, 1, 2, 512), device="cuda")
    got = kq.latent_append(P.cache, P.table, P.seq_lens, x, x[..., :64], x[:, :, 0, :].repeat(1, 1, 2)[..., :576].contiguous(), rope)
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 5
    assert torch.equal(got, torch.zeros_like(got)) and torch.equal(P.c.nan_to_num(9.0), before.nan_to_num(9.0))


# ---- the move, and all of it together

@pytest.mark.parametrize("dtype", [BF16, F8])
def test_latent_accept(dtype):
    T, lens, layers = 21, [21, 0, 64, 300], 5
    r = np.random.default_rng(3)
    Ps = [Latent(lens, 256, 32, 8, dtype, seed=70, pad=32) for _ in range(layers)]
    g = torch.Generator().manual_seed(5)
    for P in Ps:
        P.c.copy_((torch.randn(P.c.shape, generator=g) * 9).to(dtype))
    before = [P.c.clone() for P in Ps]
    masks = trees(4, T, 9)
    tokens, ids = (r.integers(0, 2, (4, T)).astype(np.int32) for _ in range(2))
    path, count, nxt, new = kq.tree_accept(kq.CacheSet([P.cache for P in Ps]), Ps[0].table, Ps[0].seq_lens, to_tensor(masks),
                                           torch.from_numpy(tokens).cuda(), torch.from_numpy(ids).cuda())
    torch.cuda.synchronize()
    table, deep = Ps[0].table.cpu().numpy(), 0
    want = [x.clone() for x in before]
    for b in range(4):
        p, n, length = walk(masks[b], lens[b], tokens[b], ids[b])
        deep = max(deep, len(p))
        assert path[b].tolist() == p + [-1] * (T - len(p))
        assert (int(count[b]), int(nxt[b]), int(new[b])) == (len(p), n, length)
        base = max(0, lens[b] - T)
        for i, u in enumerate(p):
            for x, y in zip(before, want):
                y[table[b, (base + i) // 8], (base + i) % 8] = x[table[b, (base + u) // 8], (base + u) % 8]
    assert deep > 2
    for P, y in zip(Ps, want):
        assert torch.equal(P.c.float(), y.float())


def test_a_latent_layer_step_by_step_equals_its_prompt():
    """Prompt at once against token by token, and a tree's step, captured in a graph on another stream."""
    B, H, C, R, n = 2, 16, 512, 64, 40
    g = torch.Generator().manual_seed(3)
    c, ql, qr = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((B, n, C + R), (B, n, H, C), (B, n, H, R)))
    rope = kq.RopeNorm(kq.rope_table(64, R), interleaved=True, k_norm=torch.ones(C, device="cuda"))
    P, Q = (Latent([n, n], C, R, 16, BF16, seed=4, fill="zero") for _ in range(2))
    whole = kq.latent_append(P.cache, P.table, P.seq_lens, ql, qr, c, rope)
    ws = kq.latent_attn_workspace(P.cache, B, 64, H)
    all_at_once = kq.latent_attn(P.cache, P.table, P.seq_lens, whole, ws, 0.07)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    side, out = torch.cuda.Stream(), {}

    def step():
        lens.add_(1)
        x, a, b = (y.index_select(1, at) for y in (c, ql, qr))
        q1 = kq.latent_append(Q.cache, Q.table, lens, a, b, x, rope)
        out["o"] = kq.latent_attn(Q.cache, Q.table, lens, q1, ws, 0.07)
        at.add_(1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        lens.fill_(0)
        at.fill_(0)
        for t in range(n):
            graph.replay()
            torch.cuda.synchronize()
            d = (out["o"][:, 0].float() - all_at_once[:, t].float()).abs()
            # each is within 2^-8 (sum p|c| + |out|) and a little of the same value; sum p|c| is below 4 here
            assert bool((d <= 2 * 2.0 ** -8 * (4 + all_at_once[:, t].float().abs()) + 2.0 ** -10).all())
    assert torch.equal(P.c.nan_to_num(5.0), Q.c.nan_to_num(5.0))


# ---- many items, shared workspaces, long pools, other streams

@pytest.mark.parametrize("dtype", [BF16, F8])
def test_latent_attn_more_sequences_than_ranges_and_one_split(dtype):
    """Parts joined range by range: 330 short sequences beside two that many ranges share."""
    lens = [int(x) for x in np.random.default_rng(4).integers(0, 70, 332)]
    lens[100], lens[331] = 9000, 5003
    P = Latent(lens, 256, 32, 16, dtype, seed=9)
    check_latent(P, latent_q(332, 1, 8, 288, 6))
    check_latent(P, latent_q(332, 2, 8, 288, 7), [trees(1, 2, b)[0] for b in range(332)])


@pytest.mark.parametrize("dtype,every,longer", [(BF16, 7, 400), (F8, 13, 90)])
def test_latent_attn_many_short_segments_between_longer_ones(dtype, every, longer):
    """Ranges of a dozen segments, most of one tile."""
    lens = [longer + b % 40 if b % every == 0 else 1 + b % 45 for b in range(1500)]
    P = Latent(lens, 256, 32, 16, dtype, seed=every)
    check_latent(P, latent_q(1500, 1, 3, 288, every))


def test_latent_attn_bad_vectors_in_some_of_many_segments():
    """Sequences with a vector that is not finite, which their newest token alone sees: their segments run twice, and the others
    of the range are as they are without."""
    lens = [2 + b % 70 for b in range(1100)]
    P = Latent(lens, 256, 32, 16, BF16, seed=3)
    q = latent_q(1100, 2, 3, 288, 4)
    clean = check_latent(P, q)
    hit = [b for b in range(1100) if b % 5 == 0 or 600 < b < 630]
    for b in hit:
        j = lens[b] - 1
        P.c[int(P.table[b, j // 16]), j % 16, b % 256] = float("nan")
    ws = kq.latent_attn_workspace(P.cache, 1100, 2, 3)
    out = kq.latent_attn(P.cache, P.table, P.seq_lens, q, ws, (128 + 32) ** -0.5)
    keep = torch.ones((1100, 2), dtype=torch.bool, device="cuda")
    keep[hit, 1] = False
    assert torch.equal(out[keep], clean[keep]) and out[~keep].isnan().all()


def test_latent_attn_one_workspace_for_calls_of_all_shapes():
    """In turn, on one stream, what the largest call asked for: with and without a tree, few and many rows, splits or none."""
    P = Latent([3000, 5, 0, 64, 900, 17], 512, 64, 16, BF16, seed=5)
    F = Latent([5000, 70], 512, 64, 32, F8, seed=6)
    shapes = [(P, 6, 7, 64), (P, 6, 1, 16), (F, 2, 1, 3), (P, 6, 2, 100), (F, 2, 33, 16), (P, 6, 1, 1)]
    ws = torch.zeros(max(kq.latent_attn_workspace(p.cache, b, t, h).numel() for p, b, t, h in shapes), dtype=torch.uint8,
                     device="cuda")
    for rep in range(2):
        for p, b, t, h in shapes:
            check_latent(p, latent_q(b, t, h, 576, t + h + rep), trees(b, t, h) if t > 2 else None, ws=ws)


@pytest.mark.parametrize("dtype", [BF16, F8])
def test_latent_ops_in_pages_past_2_to_the_32_bytes_and_elements(dtype):
    T, lens, page = 5, [5, 700, 33], 64
    P = Latent(lens, 512, 64, page, dtype, seed=3)
    n = P.c.shape[0]
    far = -(-(2 ** 32 + 4096) // (page * 576))
    pool = torch.empty((far + n, page, 576), dtype=dtype, device="cuda")
    pool[:far].view(torch.uint8).fill_(0xff)  # NaN
    pool[far:] = P.c
    table = torch.where(P.table >= 0, P.table + far, P.table)
    big = kq.LatentCache(pool, 512, P.scale)
    q, masks = latent_q(3, T, 16, 576, 4), trees(3, T, 5)
    ws = kq.latent_attn_workspace(P.cache, 3, T, 16)
    g = torch.Generator().manual_seed(5)
    c, ql, qr = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((3, T, 576), (3, T, 16, 512), (3, T, 16, 64)))
    rope = kq.RopeNorm(kq.rope_table(800, 64))
    words, ids = (torch.randint(0, 2, (3, T), generator=g).int().cuda() for _ in range(2))
    outs = []
    for cache, tab in ((P.cache, P.table), (big, table)):
        a = kq.latent_append(cache, tab, P.seq_lens, ql, qr, c, rope, tree=to_tensor(masks))
        o = kq.latent_attn(cache, tab, P.seq_lens, q, ws, 0.07, tree=to_tensor(masks))
        outs.append([a, o, *kq.tree_accept(kq.CacheSet([cache]), tab, P.seq_lens, to_tensor(masks), words, ids)])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert torch.equal(pool[far:].view(torch.uint8), P.c.view(torch.uint8))
    assert bool((pool[:far].view(torch.int64) == -1).all())


def test_latent_attn_rows_with_strides_on_another_stream():
    """Queries that are a slice of a wider tensor; a stream that waits for nothing else."""
    P = Latent([900, 40, 0], 512, 64, 16, BF16, seed=2)
    wide = latent_q(3, 4, 24, 576, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_latent(P, wide[:, :, 5:21], stream=side)
    check_latent(P, wide[:, :, 8:12], trees(3, 4, 1), stream=side)


@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("power", [-108, 108])
def test_latent_attn_queries_far_from_one(dtype, power):
    """Queries and a scale whose product is an ordinary one's."""
    P = Latent([700, 64, 5], 512, 64, 16, dtype, seed=2)
    check_latent(P, latent_q(3, 2, 16, 576, 3, mul=1.4 * 2.0 ** power), scale=0.07 * 2.0 ** -power)


# ---- the weights' rounding

def closely(P, q, masks=None, scale=None):
    """Weights are rounded once, and it is the rounded ones that are summed: with p_j (1 + e_j) in both sums the result is off
    by sum_j p_j e_j (c_j - out), |e_j| <= 2^-8 as bf16, 2^-11 (or 2^-29 of the row's largest weight) as fp16 beside an e4m3
    cache.  The rest as above, and the weights' fp32 sum, (n/64 + 32) 2^-24."""
    B, T, H, W = q.shape
    scale = (128 + P.R) ** -0.5 if scale is None else scale
    f8 = P.c.dtype == F8
    unit, least = (2.0 ** -11, 2.0 ** -29) if f8 else (2.0 ** -8, 0.0)
    out = kq.latent_attn(P.cache, P.table, P.seq_lens, q, kq.latent_attn_workspace(P.cache, B, T, H), scale,
                         tree=None if masks is None else to_tensor(masks))
    got, qn, square, bound = f64(out.float()), f64(q.float()), 0.0, 0.0
    for b in range(B):
        c = P.dense(b)
        for t, cols in enumerate(columns(None if masks is None else masks[b], P.lens[b], T)):
            if not cols:
                continue
            k, n = c[cols], len(cols)
            s = qn[b, t] @ k.T * scale
            ds = (W + 8) * 2.0 ** -23 * abs(scale) * np.max(np.abs(qn[b, t]) @ np.abs(k).T, axis=1)[:, None]
            p = np.exp(s - s.max(1, keepdims=True))
            weights = p.sum(1, keepdims=True)
            v = k[:, :P.C]
            ref, sv = p @ v / weights, p @ np.abs(v) / weights
            off = np.abs(v[None] - ref[:, None])  # |c_j - out|
            spread = (np.einsum("hj,hjd->hd", p, off) * unit + least * off.sum(1)) / weights
            rest = 2 * ds + 2.0 ** -20 + (n / 8 + 128) * 2.0 ** -23 + (n / 64 + 32) * 2.0 ** -24
            err = np.abs(got[b, t] - ref)
            tol = (spread + rest * sv) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(ref)
            assert np.all(np.isfinite(err)) and np.all(err <= tol), (b, t, float(np.nanmax(err / tol)))
            square += (err ** 2).sum()
            # of a rounding to bf16, a step of up to 2^-7 of the value: step / sqrt(12) in the mean square
            bound += ((2.0 ** -8 / 3 ** 0.5 * np.abs(ref) + spread + rest * sv) ** 2).sum()
    assert square <= bound, (square / bound) ** 0.5


@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("C,R,T,H,tree", [(512, 64, 1, 16, False), (256, 32, 1, 40, False), (512, 64, 9, 16, True), (512, 32, 3, 5, False)])
def test_latent_attn_rounds_each_weight_once(dtype, C, R, T, H, tree):
    lens = [700, T, 90, 0, 333]
    P = Latent(lens, C, R, 16, dtype, seed=C + H)
    closely(P, latent_q(5, T, H, C + R, T + H), trees(5, T, T + 2) if tree else None)


@pytest.mark.parametrize("dtype,n,per_sm", [(BF16, 64, 2), (BF16, 500, 1), (F8, 64, 2)])
@pytest.mark.parametrize("late", [33, 50, 63])
def test_latent_attn_a_late_position_that_dominates(dtype, n, per_sm, late):
    """A position behind the first tile, by powers of two (that are not whole numbers) which do not raise the row's maximum: its
    weight is any number, and that number's rounding is not the result's.  As many sequences as leave each one whole."""
    B = per_sm * torch.cuda.get_device_properties(0).multi_processor_count
    P = Latent([n] * B, 512, 64, 16, dtype, seed=late)
    j = torch.arange(n, device="cuda")
    pages = P.table.long()[:, j // 16]
    P.c[pages, j % 16, 512] = torch.zeros((B, n), device="cuda").to(dtype)
    P.c[pages[:, late], late % 16, 512] = torch.full((B,), 1 / P.scale, device="cuda").to(dtype)
    most = 10.9 if dtype == F8 else 23.9
    q = torch.zeros((B, 1, 6, 576), device="cuda")
    q[..., 512] = (torch.linspace(0.5, 1.0, 6 * B, device="cuda") * most * 0.6931471805599453).view(B, 1, 6)
    closely(P, q.to(BF16), scale=1.0)


# ---- as many rows as a call takes

@pytest.mark.parametrize("dtype,T,H", [(BF16, 64, 256), (F8, 64, 256), (BF16, 38, 256), (BF16, 59, 163), (F8, 19, 256), (BF16, 64, 119)])
def test_latent_attn_as_many_row_tiles_as_sms_and_more(dtype, T, H):
    """256, 152, 151 (no tile, or next to none, is left over by all of them side by side), 76 and 119 row tiles."""
    lens = [T + 45, T, 3]
    P = Latent(lens, 256, 32, 16, dtype, seed=T)
    check_latent(P, latent_q(3, T, H, 288, T), [chain(T), trees(1, T, T)[0], trees(1, T, T + 1)[0]])


# ---- from the products on

@pytest.mark.parametrize("qtype,T,H", [(1, 1, 16), (3, 4, 20), (1, 4, 128)])
def test_a_latent_layer_from_its_quantized_products(qtype, T, H):
    """Queries absorbed by kq_moe_matvec, whose experts are the heads, then append, attention and each head's values by
    kq_moe_matvec again: against attention over expanded keys and values in 64 bits.  An absorbed query is off by 2^-8 of
    itself (its bf16) and a product's bound (tests/gpu_util.py); a score so by scale times that over sum |c|, twice that in
    the weights, with 2^-8 for their rounding; then the result's bf16 and the values' product."""
    C, R, N, B, page = 512, 64, 128, 512 // (T * H) if T * H > 64 else 2, 16
    g, t = synth.rng(77, qtype, T, H), torch.Generator().manual_seed(H)
    up, down = synth.gen_matrix(qtype, H * C, N, g), synth.gen_matrix(qtype, H * N, C, g)  # [C, N] and [N, C] per head
    dense = []
    for w, rows, cols in ((up, H * C, N), (down, H * N, C)):
        full = -(-cols // 256) * 256
        y = torch.empty(rows * full, device="cuda")
        w = torch.from_numpy(w).cuda()
        kq.kq_dequant(qtype, w, y, rows * full)
        dense.append((w, f64(y.view(rows, full)[:, :cols]).reshape(H, -1, cols)))
    lens = [T + 57 * b for b in range(B)]
    P = Latent(lens, C, R, page, BF16, seed=H)
    ids = torch.arange(H, dtype=torch.int32, device="cuda").repeat(B * T, 1)

    def heads(w, x, n, k):
        y = torch.empty((B * T, H, n), device="cuda")
        ws = kq.moe_workspace(n, B * T, H, H)
        kq.kq_moe_matvec(qtype, w, H, ids, None, x.reshape(B * T, H, k).contiguous(), kq.KQ_BF16, True, y, n, k, B * T, H, ws, ws.numel())
        kq.kq_moe_check(ws)
        return y.view(B, T, H, n)
    q = torch.randn((B, T, H, N + R), generator=t).to(BF16).cuda()  # a query product's rows
    c = torch.randn((B, T, C + R), generator=t).cuda()
    rope = kq.RopeNorm(kq.rope_table(max(lens) + 1, R), k_norm=torch.ones(C, device="cuda"))
    absorbed = heads(dense[0][0], q[..., :N], C, N)
    a = kq.latent_append(P.cache, P.table, P.seq_lens, absorbed, q[..., N:].float(), c, rope)
    size = float(absorbed.square().mean().sqrt())
    scale = 1.0 / (size * C ** 0.5)  # scores about one
    o = kq.latent_attn(P.cache, P.table, P.seq_lens, a, kq.latent_attn_workspace(P.cache, B, T, H), scale)
    y = f64(heads(dense[1][0], o, N, C))
    A, V, qn, an = dense[0][1], dense[1][1], f64(q[..., :N].float()), f64(a.float())
    for b in range(B):
        cc = P.dense(b)
        for i in range(T):
            k = cc[:lens[b] - T + i + 1]
            lat, rot = k[:, :C], an[b, i, :, C:] @ k[:, C:].T      # (the rotated part is tested above)
            keys = np.einsum("hcn,jc->hjn", A, lat)                # expanded
            s = (np.einsum("hn,hjn->hj", qn[b, i], keys) + rot) * scale
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            latents = p @ lat
            ref = np.einsum("hnc,hc->hn", V, latents)
            dq = 2.0 ** -8 * np.abs(an[b, i, :, :C]) * (1 + 2.0 ** -8) + TOL["bf16"] * np.einsum("hcn,hn->hc", np.abs(A), np.abs(qn[b, i]))
            ds = scale * (dq @ np.abs(lat).T).max(1)[:, None] + 2.0 ** -12
            sv = p @ np.abs(lat)
            do = (np.expm1(2 * ds) + 2.0 ** -7) * sv + 2.0 ** -8 * np.abs(latents)
            tol = np.einsum("hnc,hc->hn", np.abs(V), do + TOL["bf16"] * (np.abs(latents) + do))
            err = np.abs(y[b, i] - ref)
            assert np.all(err <= tol), (b, i, float((err / tol).max()))
            # far within it, as the errors are independent: their root mean square is below a tenth of the values'
            assert (err ** 2).mean() <= 0.01 * (ref ** 2).mean(), (b, i)
