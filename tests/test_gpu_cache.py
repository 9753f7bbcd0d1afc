"""kq_kv_append and kq_attn_decode against their definitions in 64 bits.

Bounds (derived, per element):
append.  The norm's factor carries the rounding of a D-term fp32 sum of
squares (8 terms a lane, then a tree: below 16 ulps), rsqrt's 2 ulps and three
products; a rotation adds two products and a sum: together below 2^-20 of
|a| + |b|, the rotation partners after the norm.  Then one rounding: 2^-24
(fp32), 2^-8 (bf16: 8 significant bits), 2^-4 or half of the subnormal step
2^-9 (e4m3), of the stored value.
attention.  A score is a D-term fp32 sum of exact products (the tensor cores
may truncate: 2^-23 a step) with a few roundings for scale and cap, so
|ds| <= (D + 8) 2^-23 scale sum|q k| + cap 2^-21 and the weights' relative
error is 2 max|ds| + 2^-20 (exp).  Weights enter the second product in 16-bit
parts, 2^-16 relative for bf16 q and 2^-20 for fp32 q, and the sums over n
positions add at most (n/8 + 128) 2^-23.  All of it multiplies
sum_j p_j |v_j|; then one rounding of the result, 2^-8 (bf16) or 2^-24.
"""
import math

import numpy as np
import pytest
import torch

from gguf_quant_weight_super_gb300 import kq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F8, F32 = torch.bfloat16, torch.float8_e4m3fn, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    require_gpu()
    from gguf_quant_weight_super_gb300 import build
    build.build()
    kq.lib()
    kq.kq_device_error(clear=True)
    yield
    assert kq.kq_device_error() == 0


def f64(t):
    return t.double().cpu().numpy()


class Paged:
    """A cache of random values whose pages lie in any order, with lengths; slots no sequence has hold NaN."""

    def __init__(self, lens, Hkv, D, page, dtype, seed, layout="token", spare=2, fill="random"):
        g = torch.Generator().manual_seed(seed)
        self.lens = list(lens)
        B = len(self.lens)
        used = [-(-max(0, n) // page) for n in self.lens]
        n_pages = sum(used) + spare
        W = max(1, max(used, default=1)) + 1
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        table = torch.full((B, W), -7, dtype=torch.int32)  # entries past a length are never read
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = perm[at:at + u]
            at += u
        shape = (n_pages, page, Hkv, D) if layout == "token" else (n_pages, Hkv, page, D)
        pools = []
        for _ in range(2):
            x = torch.randn(shape, generator=g)
            pools.append(x if fill == "random" else torch.zeros(shape))
        seen = torch.zeros((n_pages, page), dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for i in range(used[b]):
                seen[table[b, i], :min(page, n - i * page)] = True
        mask = seen[:, :, None, None] if layout == "token" else seen[:, None, :, None]
        pools = [torch.where(mask, x, float("nan")).cuda() for x in pools]
        self.k_scale, self.v_scale = (0.25, 0.5) if dtype == F8 else (1.0, 1.0)
        k, v = ((p / s).to(dtype) for p, s in zip(pools, (self.k_scale, self.v_scale)))
        if layout == "head":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        self.k, self.v, self.table, self.page = k, v, table.cuda(), page
        self.cache = kq.KVCache(k, v, self.k_scale, self.v_scale)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()

    def dense(self, b):
        """k, v [len, Hkv, D] of a sequence in 64 bits."""
        n = max(0, self.lens[b])
        j = np.arange(n)
        pages = self.table[b].cpu().numpy()[j // self.page]
        return (f64(self.k.float())[pages, j % self.page] * self.k_scale,
                f64(self.v.float())[pages, j % self.page] * self.v_scale)


def attn_ref(P, q, scale, cap, window):
    """(out, bound's sum p|v|, max|ds| bound) per element in 64 bits."""
    q = f64(q.float())
    B, T, Hq, D = q.shape
    out, sv, ds = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, T, Hq, 1))
    for b in range(B):
        k, v = P.dense(b)
        Hkv = k.shape[1]
        for t in range(T):
            pos = P.lens[b] - T + t
            if pos < 0:
                continue
            lo = max(0, pos - window + 1) if window else 0
            for h in range(Hq):
                kk, vv = k[lo:pos + 1, h * Hkv // Hq], v[lo:pos + 1, h * Hkv // Hq]
                s = kk @ q[b, t, h] * scale
                ds[b, t, h] = (D + 8) * 2.0 ** -23 * abs(scale) * np.max(np.abs(kk) @ np.abs(q[b, t, h])) + cap * 2.0 ** -21
                if cap:
                    s = cap * np.tanh(s / cap)
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, t, h], sv[b, t, h] = p @ vv, p @ np.abs(vv)
    return out, sv, ds


def check_attn(P, q, scale=None, cap=0.0, window=0, stream=None):
    B, T, Hq, D = q.shape
    ws = kq.attn_workspace(P.cache, B, T, Hq)
    out = torch.full((B, T, Hq, D), float("nan"), dtype=q.dtype, device="cuda")
    kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, scale=scale, softcap=cap, window=window, out=out, stream=stream)
    torch.cuda.synchronize()
    ref, sv, ds = attn_ref(P, q, D ** -0.5 if scale is None else scale, cap, window)
    n = max(1, max(P.lens))
    part, rnd = (2.0 ** -16, 2.0 ** -8) if q.dtype == BF16 else (2.0 ** -20, 2.0 ** -24)
    d = 2 * ds + 2.0 ** -20 + part + (n / 8 + 128) * 2.0 ** -23
    tol = d * sv * (1 + rnd) + rnd * np.abs(ref)
    err = np.abs(f64(out.float()) - ref)
    assert np.all(np.isfinite(err)) and np.all(err <= tol), float(np.nanmax(err / np.maximum(tol, 1e-300)))
    again = torch.empty_like(out)
    kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, scale=scale, softcap=cap, window=window, out=again)
    torch.cuda.synchronize()
    assert torch.equal(again, out)  # the same bits again, on a workspace that was used
    return out


def rand_q(B, T, Hq, D, dtype, seed, mul=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, T, Hq, D), generator=g) * mul).to(dtype).cuda()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("qt", [BF16, F32])
@pytest.mark.parametrize("T,G", [(1, 4), (3, 1), (7, 5)])
def test_attn_matches_definition(D, dtype, qt, T, G):
    P = Paged([1, 700, 33, 64], 2, D, 16, dtype, seed=D + T + G)
    check_attn(P, rand_q(4, T, 2 * G, D, qt, 5))


@pytest.mark.parametrize("T,Hkv,G", [(1, 1, 1), (1, 3, 2), (1, 2, 16), (2, 1, 8), (4, 2, 4), (5, 1, 7), (16, 1, 1),
                                     (16, 2, 4), (16, 1, 8), (15, 1, 9), (16, 1, 16)])
def test_attn_head_groups_and_blocks(T, Hkv, G):
    P = Paged([517, 100, 16], Hkv, 128, 32, BF16, seed=T * G)
    check_attn(P, rand_q(3, T, Hkv * G, 128, BF16, 6))


@pytest.mark.parametrize("page", [1, 2, 8, 64, 256, 1024])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_attn_pages_and_layouts(page, layout):
    P = Paged([777, 1, 63, 65, 256], 2, 128, page, BF16, seed=page, layout=layout)
    check_attn(P, rand_q(5, 2, 6, 128, BF16, 7))


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 191, 4000])
@pytest.mark.parametrize("T", [1, 4])
def test_attn_lengths(n, T):
    P = Paged([n], 1, 64, 16, BF16, seed=n)
    check_attn(P, rand_q(1, T, 4, 64, BF16, 8))


@pytest.mark.parametrize("T", [1, 16])
def test_attn_empty_and_padding_rows_are_zero(T):
    P = Paged([0, 5, 0, 40, 0], 2, 128, 16, BF16, seed=3)
    out = check_attn(P, rand_q(5, T, 8, 128, BF16, 9))
    assert torch.all(out[0] == 0) and torch.all(out[2] == 0) and torch.all(out[4] == 0)
    if T == 16:
        assert torch.all(out[1, :11] == 0) and torch.all(out[1, 11:].abs().sum(-1) > 0)
    P = Paged([0, 0], 2, 128, 16, BF16, seed=3)
    assert torch.all(check_attn(P, rand_q(2, T, 8, 128, BF16, 9)) == 0)


@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 5000])
@pytest.mark.parametrize("T,cap,dtype", [(1, 0.0, BF16), (1, 30.0, F8), (6, 20.0, BF16), (16, 0.0, BF16)])
def test_attn_window_and_softcap(window, T, cap, dtype):
    P = Paged([300, 90, 12, 1030], 2, 128, 32, dtype, seed=window)
    check_attn(P, rand_q(4, T, 4, 128, BF16, 10), cap=cap, window=window)


@pytest.mark.parametrize("qt", [BF16, F32])
def test_attn_large_scores(qt):
    """Scores of hundreds: one position takes nearly all of the weight."""
    P = Paged([900, 257], 2, 128, 16, BF16, seed=11)
    check_attn(P, rand_q(2, 1, 8, 128, qt, 12, mul=60.0))


def test_attn_negative_scale_and_equal_scores():
    P = Paged([333], 1, 64, 16, BF16, seed=12)
    check_attn(P, rand_q(1, 2, 2, 64, BF16, 13), scale=-0.2)
    check_attn(P, rand_q(1, 2, 2, 64, BF16, 13), scale=0.0)


@pytest.mark.parametrize("what", ["v_nan", "k_nan", "v_inf"])
@pytest.mark.parametrize("qt", [BF16, F32])
def test_attn_unseen_positions_do_not_matter(what, qt):
    """A position that some tokens of the block do not see (later ones, and ones that left the window) has no
    influence on them, whatever it holds; the tokens that see it get what it gives."""
    T, n, window = 8, 200, 64
    P = Paged([n, 64], 2, 128, 16, BF16, seed=14)
    q = rand_q(2, T, 8, 128, qt, 15)
    ws = kq.attn_workspace(P.cache, 2, T, 8)
    clean = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window)
    bad = float("inf") if what == "v_inf" else float("nan")
    pool = P.k if what == "k_nan" else P.v
    late, early = n - 3, n - T - window + 3  # seen by tokens t >= 5; by tokens t <= 2
    for pos in (late, early):
        pool[int(P.table[0, pos // 16]), pos % 16, 0, 3] = bad
    got = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window)
    torch.cuda.synchronize()
    for t in range(T):
        sees = t >= 5 or t <= 2
        if not sees:
            assert torch.equal(got[0, t], clean[0, t]), t
        elif what == "k_nan":
            assert torch.all(torch.isnan(got[0, t, :4])), t
            assert torch.equal(got[0, t, 4:], clean[0, t, 4:]), t
        else:
            hit = got[0, t, :4, 3].float()
            assert torch.all(torch.isnan(hit) if what == "v_nan" else torch.isinf(hit)), t
            rest = [d for d in range(128) if d != 3]
            assert torch.equal(got[0, t][:, rest], clean[0, t][:, rest]), t
            assert torch.equal(got[0, t, 4:], clean[0, t, 4:]), t
    assert torch.equal(got[1], clean[1])


def test_attn_query_rows_at_a_stride():
    P = Paged([100, 45], 2, 128, 16, BF16, seed=16)
    buf = rand_q(2, 3, 12, 128, BF16, 17)
    q = buf[:, :, :8]  # rows of a fused buffer
    ws = kq.attn_workspace(P.cache, 2, 3, 8)
    a = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws)
    b = kq.attn_decode(P.cache, P.table, P.seq_lens, q.contiguous(), ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_attn_many_sequences():
    g = np.random.default_rng(1)
    lens = [int(x) for x in g.integers(0, 90, 300)]
    P = Paged(lens, 1, 64, 8, BF16, seed=18)
    check_attn(P, rand_q(300, 1, 2, 64, BF16, 19))


def test_attn_on_another_stream_and_in_a_graph():
    P = Paged([3000, 10], 2, 128, 16, BF16, seed=20)
    q = rand_q(2, 1, 8, 128, BF16, 21)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    check_attn(P, q, stream=s)
    ws = kq.attn_workspace(P.cache, 2, 1, 8)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, out=out)
    want = kq.attn_decode(P.cache, P.table, P.seq_lens, q, kq.attn_workspace(P.cache, 2, 1, 8))
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_attn_long_cache_past_32_bits():
    """Element offsets past 2^32: a pool whose last pages start there."""
    D, Hkv, page = 128, 8, 64
    n_pages = (1 << 32) // (D * Hkv * page) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 2 * 2 * n_pages * page * Hkv * D + (8 << 30):
        pytest.skip("not enough device memory")
    k = torch.empty((n_pages, page, Hkv, D), dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    n = 2000
    u = -(-n // page)
    P = Paged([n], Hkv, D, page, BF16, seed=22)
    table = torch.arange(n_pages - u, n_pages, dtype=torch.int32, device="cuda").flip(0).view(1, u).contiguous()
    k[table[0].long()] = P.k[P.table[0, :u].long()]
    v[table[0].long()] = P.v[P.table[0, :u].long()]
    q = rand_q(1, 1, 32, D, BF16, 23)
    ws = kq.attn_workspace(P.cache, 1, 1, 32)
    want = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws)
    got = kq.attn_decode(kq.KVCache(k, v), table, P.seq_lens, q, ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    # the writer reaches the same pages
    x = rand_q(1, 1, 32, D, BF16, 24)
    kv = rand_q(1, 1, Hkv, D, BF16, 25)
    kq.kv_append(kq.KVCache(k, v), table, P.seq_lens, x, kv, kv, kq.RopeNorm())
    torch.cuda.synchronize()
    at = int(table[0, (n - 1) // page])
    assert torch.equal(k[at, (n - 1) % page], kv[0, 0]) and torch.equal(v[at, (n - 1) % page], kv[0, 0])


def test_bad_pages_and_lengths_are_recorded():
    P = Paged([40, 50], 2, 64, 16, BF16, seed=26)
    q = rand_q(2, 1, 4, 64, BF16, 27)
    ws = kq.attn_workspace(P.cache, 2, 1, 4)
    good = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws)
    for bad_id in (-1, P.k.shape[0], 1 << 30):
        table = P.table.clone()
        table[0, 1] = bad_id
        got = kq.attn_decode(P.cache, table, P.seq_lens, q, ws)
        torch.cuda.synchronize()
        assert kq.kq_device_error(clear=True) == 4
        assert torch.equal(got[1], good[1])
    lens = P.seq_lens.clone()
    lens[0] = P.table.shape[1] * 16 + 1
    table = P.table.clone()
    table[0, :] = table[1, 0]
    got = kq.attn_decode(P.cache, table, lens, q, ws)
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 4
    assert torch.equal(got[1], good[1])
    kv = rand_q(2, 1, 2, 64, BF16, 28)
    before = P.k.clone()
    kq.kv_append(P.cache, table, lens, q, kv, kv, kq.RopeNorm())     # past the table
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 4
    table = P.table.clone()
    table[0, 39 // 16] = 1 << 30
    kq.kv_append(P.cache, table, P.seq_lens, q, kv, kv, kq.RopeNorm())
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 4
    rope = kq.RopeNorm(kq.rope_table(45, 64))                          # position 49 is outside
    out = kq.kv_append(P.cache, P.table, P.seq_lens, q, kv, kv, rope)
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 5
    assert torch.all(out[1] == 0) and torch.any(out[0] != 0)
    changed = (P.k.view(torch.int16) != before.view(torch.int16)).any(-1).any(-1).sum().item()
    assert changed == 2  # the two sequences' last slots only


# ---------------------------------------------------------------------------
# kv_append
# ---------------------------------------------------------------------------

def append_case(lens, T, Hq, Hkv, D, page, xt, qt, ct, seed, rot=None, inter=False, norm=True, off=0.0, fused=False,
                layout="token", mul=1.5):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    P = Paged(lens, Hkv, D, page, ct, seed, layout=layout, fill="zero")
    x = (torch.randn((B, T, Hq + 2 * Hkv, D), generator=g) * mul).to(xt).cuda()
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rot = D if rot is None else rot
    cs = kq.rope_table(max(1, max(lens)), rot, base=1e6) if rot else None
    wq, wk = ((1.0 - off + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2)) if norm else (None, None)
    rope = kq.RopeNorm(cs, interleaved=inter, q_norm=wq, k_norm=wk, eps=1e-6, norm_offset=off)
    q_out = torch.full((B, T, Hq, D), float("nan"), dtype=qt, device="cuda")
    before = (f64(P.k.float()), f64(P.v.float()))
    kq.kv_append(P.cache, P.table, P.seq_lens, q, k, v, rope, q_out=q_out)
    torch.cuda.synchronize()

    def turned(x, w, b, t, pos):
        """(value, |a| + |b|) of one token's heads."""
        y = f64(x.float())[b, t]
        if w is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6) * (f64(w) + off)
        size = np.abs(y)
        if rot:
            c, s = (f64(cs)[pos, :rot // 2], f64(cs)[pos, rot // 2:])
            i = np.arange(rot // 2)
            i, j = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            z = y.copy()
            z[:, i], z[:, j] = y[:, i] * c - y[:, j] * s, y[:, j] * c + y[:, i] * s
            size[:, i] = size[:, j] = size[:, i] + size[:, j]
            y = z
        return y, size

    def near(got, want, size, dtype):
        e = 2.0 ** -20 * size
        if dtype == F8:
            want = np.clip(want, -448, 448)
            tol = e * 1.1 + np.maximum(2.0 ** -4 * np.abs(want) * 1.01, 2.0 ** -10)
        else:
            rnd = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
            tol = e * (1 + rnd) + rnd * np.abs(want)
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))

    gk, gv, gq = f64(P.k.float()), f64(P.v.float()), f64(q_out.float())
    touched = np.zeros(gk.shape[:2], bool)
    for b, n in enumerate(lens):
        for t in range(T):
            pos = n - T + t
            if pos < 0:
                assert np.all(gq[b, t] == 0)
                continue
            y, size = turned(q, wq, b, t, pos)
            near(gq[b, t], y, size, qt)
            at = (int(P.table[b, pos // page]), pos % page)
            touched[at] = True
            y, size = turned(k, wk, b, t, pos)
            near(gk[at], y / P.k_scale, size / P.k_scale, ct)
            y = f64(v.float())[b, t] / P.v_scale
            near(gv[at], y, np.abs(y), ct)
    for got, old in ((gk, before[0]), (gv, before[1])):  # nothing else changed
        assert np.array_equal(got[~touched], old[~touched], equal_nan=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("xt,qt,ct", [(F32, BF16, BF16), (BF16, BF16, BF16), (F32, F32, F8), (BF16, F32, F8),
                                      (F32, BF16, F8), (BF16, F32, BF16)])
@pytest.mark.parametrize("inter", [False, True])
def test_append_matches_definition(D, xt, qt, ct, inter):
    append_case([1, 300, 17], 1, 6, 2, D, 16, xt, qt, ct, seed=D, inter=inter)


@pytest.mark.parametrize("T", [1, 2, 5, 33])
@pytest.mark.parametrize("page", [1, 8, 64])
@pytest.mark.parametrize("fused", [False, True])
def test_append_blocks_pages_and_fused_rows(T, page, fused):
    """Lengths below T leave padding tokens; an empty sequence has nothing else."""
    append_case([100, 3, 0, T, T + 1], T, 3, 1, 128, page, BF16, BF16, BF16, seed=T + page, fused=fused, off=1.0)


@pytest.mark.parametrize("rot", [0, 8, 24, 64, 104, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_part_of_the_head(rot, inter, norm):
    append_case([50, 9], 3, 5, 2, 128, 16, F32, BF16, BF16, seed=rot, rot=rot, inter=inter, norm=norm)


def test_append_head_major_pages_and_far_positions():
    append_case([5000, 131072], 2, 4, 2, 64, 64, F32, F32, BF16, seed=1, layout="head")


def test_append_8bit_saturates_and_keeps_nan():
    P = Paged([1], 1, 64, 16, F8, seed=2, fill="zero")
    x = torch.zeros((1, 1, 1, 64), device="cuda")
    x[..., 0], x[..., 1], x[..., 2], x[..., 3] = 1e6, -1e6, float("nan"), float("inf")
    kq.kv_append(P.cache, P.table, P.seq_lens, x, x, x, kq.RopeNorm())
    torch.cuda.synchronize()
    k = P.k[int(P.table[0, 0]), 0, 0].float()
    assert k[0] == 448 and k[1] == -448 and torch.isnan(k[2]) and k[3] == 448 and torch.all(k[4:] == 0)


def test_rope_table_scaling():
    t = kq.rope_table(9, 8, base=100.0, factor=4.0)
    a = np.arange(9)[:, None] * 100.0 ** (-np.arange(0, 8, 2) / 8) / 4
    np.testing.assert_allclose(f64(t), np.concatenate([np.cos(a), np.sin(a)], 1), atol=1e-7)
    # by parts: fast pairs keep their frequency, slow ones are stretched
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    t = f64(kq.rope_table(2, 64, factor=8.0, trained=4096, low=1.0, high=4.0))
    got = np.arctan2(t[1, 32:], t[1, :32])
    turns = 4096 * f / (2 * math.pi)
    np.testing.assert_allclose(got[turns >= 4], f[turns >= 4], rtol=1e-5)
    np.testing.assert_allclose(got[turns <= 1], f[turns <= 1] / 8, rtol=1e-3, atol=1e-7)
    assert np.all((got <= f * (1 + 1e-3) + 1e-7) & (got >= f / 8 * (1 - 1e-3) - 1e-7))


def test_append_then_attend_is_a_decode_loop():
    """Token by token, the cache that kv_append fills gives what a dense computation gives."""
    B, Hq, Hkv, D, page, steps = 2, 4, 2, 64, 8, 20
    g = torch.Generator().manual_seed(3)
    x = torch.randn((steps, B, 1, Hq + 2 * Hkv, D), generator=g).cuda()
    k = torch.full((8, page, Hkv, D), float("nan"), dtype=BF16, device="cuda")
    v = k.clone()
    cache = kq.KVCache(k, v)
    table = torch.tensor([[5, 1, 7], [0, 2, 4]], dtype=torch.int32, device="cuda")
    rope = kq.RopeNorm(kq.rope_table(steps, D))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = kq.attn_workspace(cache, B, 1, Hq)
    outs, qs = [], []
    for i in range(steps):
        lens += 1
        q = kq.kv_append(cache, table, lens, x[i, :, :, :Hq], x[i, :, :, Hq:Hq + Hkv], x[i, :, :, Hq + Hkv:], rope)
        outs.append(kq.attn_decode(cache, table, lens, q, ws))
        qs.append(q)
    torch.cuda.synchronize()
    for i in (0, 7, 8, steps - 1):
        for b in range(B):
            j = np.arange(i + 1)
            pg = table[b].cpu().numpy()[j // page]
            kk, vv = f64(k.float())[pg, j % page], f64(v.float())[pg, j % page]
            np.testing.assert_allclose(vv, f64(x[:i + 1, b, 0, Hq + Hkv:].to(BF16).float()))
            for h in range(Hq):
                s = kk[:, h // 2] @ f64(qs[i].float())[b, 0, h] * D ** -0.5
                p = np.exp(s - s.max())
                o = (p / p.sum()) @ vv[:, h // 2]
                sv = (p / p.sum()) @ np.abs(vv[:, h // 2])
                assert np.all(np.abs(f64(outs[i].float())[b, 0, h] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -14 * sv)


@pytest.mark.parametrize("T,G,dtype", [(1, 1, BF16), (16, 2, BF16), (8, 4, F8)])
def test_attn_one_head_over_every_range(T, G, dtype):
    """One head's long cache: all the device's CTAs, and the left-over ranges, hold a part of the same item."""
    P = Paged([150001], 1, 64, 64, dtype, seed=29)
    check_attn(P, rand_q(1, T, G, 64, BF16, 30))


@pytest.mark.parametrize("dtype", [BF16, F8])
def test_attn_fp32_long_sums_keep_their_digits(dtype):
    """Values of one sign over a long cache: every step adds to the same sum.  fp32 q and out keep 2^-19 (the weights'
    parts 2^-20, a few rounded additions per step of sums that are joined from short ones)."""
    P = Paged([40000], 1, 64, 64, dtype, seed=31)
    P.v.copy_((P.v.float().nan_to_num(0.0).abs() + 0.5).to(dtype))
    q = rand_q(1, 1, 2, 64, F32, 32, mul=0.5)
    out = kq.attn_decode(P.cache, P.table, P.seq_lens, q, kq.attn_workspace(P.cache, 1, 1, 2))
    torch.cuda.synchronize()
    ref, _, _ = attn_ref(P, q, 64 ** -0.5, 0.0, 0)
    assert np.max(np.abs(f64(out) / ref - 1)) <= 2.0 ** -19
