"""kq_sample against its definition in 64 bits.

The token is exact: u is put in the middle of a word's interval, and only
words whose share is at least 2^-16 are aimed at, so that u's fp32 rounding
(2^-24) and the weights' error cannot reach an edge; top_p likewise lies in
the middle of a word's weight.  probs: w_i = exp(z), z = (l - l_max)/t carries
two fp32 roundings (|z| <= 64 here: 2^-17 in exp's argument at worst, 2^-22
near the words that are chosen, |z| <= 12: 2^-19) and exp 2 ulps, and so do
the weights it is divided by: 2^-17 relative.
"""
import numpy as np
import pytest
import torch

from gguf_quant_weight_super_gb300 import kq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    require_gpu()
    from gguf_quant_weight_super_gb300 import build
    build.build()
    kq.lib()


def ranked(row):
    """Words in descending order (ties by index; NaN as -inf) and their logits, fp64."""
    l = np.where(np.isnan(row), -np.inf, row.astype(np.float64))
    order = np.argsort(-l, kind="stable")
    return order, l[order]


def weights(l, t):
    if not t > 0:
        w = np.zeros(len(l))
        w[0] = 1.0
        return w
    z = np.full(len(l), -np.inf)
    z[l == l[0]] = 0.0
    fin = np.isfinite(l) & (l != l[0])
    if np.isfinite(l[0]):
        z[fin] = (l[fin] - l[0]) / t
    return np.exp(z)


def kept(w, k, p, mp):
    n = len(w)
    if k > 0:
        n = min(n, k)
    if p < 1:
        c = np.cumsum(w[:n])
        n = max(1, int(np.sum(c - w[:n] < p * c[-1])))
    return max(1, min(n, int(np.sum(w >= mp))))


def check(x, t, k, p, mp, aim, seed=0):
    """Rows x [M, V]; p per row may be ('mid', j): the middle of the j-th word's weight after top_k.  aim: a rank per
    row, moved to the nearest word with a share of at least 2^-16."""
    M, V = x.shape
    xs = x.float().cpu().numpy()
    u, ids, probs, ps = [], [], [], []
    for m in range(M):
        order, l = ranked(xs[m])
        w = weights(l, t[m])
        kk = 1 if not t[m] > 0 else k[m]
        pm = p[m]
        if isinstance(pm, tuple):
            c = np.cumsum(w[:kk] if kk > 0 else w)
            j = min(pm[1], len(c) - 1)
            pm = (c[j] - 0.5 * w[j]) / c[-1]
        n = kept(w, kk, pm, mp[m])
        c = np.cumsum(w[:n])
        r = min(aim[m], n - 1)
        while r > 0 and w[r] / c[-1] < 2.0 ** -16:
            r -= 1
        u.append((c[r] - 0.5 * w[r]) / c[-1])
        ids.append(order[r])
        probs.append(w[r] / c[-1])
        ps.append(pm)
    f = lambda v, dt=F32: torch.tensor(np.array(v), dtype=dt, device="cuda")  # noqa: E731
    ws = kq.sample_workspace(M, V)
    args = dict(temperature=f(t), top_k=f(k, torch.int32), top_p=f(ps), min_p=f(mp), workspace=ws)
    got, gp = kq.sample(x, f(u), **args)
    again, ap = kq.sample(x, f(u), **args)
    torch.cuda.synchronize()
    assert got.cpu().numpy().tolist() == [int(i) for i in ids]
    np.testing.assert_allclose(gp.double().cpu().numpy(), probs, rtol=2.0 ** -17)
    assert torch.equal(got, again) and torch.equal(gp, ap)
    return got


def logits(M, V, seed, dtype=F32, sd=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, V), generator=g) * sd
    top = torch.randint(0, V, (M, 24), generator=g)
    x.scatter_add_(1, top, 3.0 + 7.0 * torch.rand((M, 24), generator=g))
    return x.to(dtype).cuda()


@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 1000, 1024, 1025, 8191, 151936, 262144])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_vocabularies(V, dtype):
    M = 6
    x = logits(M, V, V, dtype)
    check(x, [0.7, 1.0, 1.3, 0.0, 1.0, 0.5], [20, 0, 0, 5, 1, 40], [1.0, ("mid", 9), 1.0, 0.5, 0.9, ("mid", 3)],
          [0.0, 0.0, 0.05, 0.0, 0.0, 0.01], [3, 5, 2, 7, 4, 1])


@pytest.mark.parametrize("k", [1, 2, 7, 50, 257, 1000, 5000, 200000])
def test_sample_top_k(k):
    x = logits(4, 20001, k, sd=1.0)
    for aim in (0, k // 2, k - 1, 10 ** 9):
        check(x, [1.0, 2.0, 0.9, 3.0], [k] * 4, [1.0] * 4, [0.0] * 4, [aim] * 4)


@pytest.mark.parametrize("j", [0, 1, 10, 500, 15000])
def test_sample_top_p(j):
    """Cuts in the likely words, in the bulk and in the tail, alone and after top_k."""
    x = logits(4, 20001, j, sd=1.0)
    for aim in (0, j, j // 2):
        check(x, [1.0, 2.0, 1.5, 1.0], [0, 0, 16000, 600], [("mid", j)] * 4, [0.0] * 4, [aim] * 4)


@pytest.mark.parametrize("mp", [0.001, 0.03, 0.5, 1.0])
def test_sample_min_p(mp):
    x = logits(3, 5000, 3)
    check(x, [1.0, 1.4, 0.8], [0, 100, 0], [1.0, 1.0, ("mid", 30)], [mp] * 3, [2, 30, 1000])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_equal_logits_go_by_index(dtype):
    V = 3001
    x = torch.full((6, V), 1.5, dtype=dtype, device="cuda")
    x[1, 100:] = 0.5                        # 100 equal leaders
    x[2, ::3] = 2.0                         # every third
    x[3, :] = 0.0
    x[3, 1::2] = -0.0                       # -0 equals 0
    check(x, [1.0] * 6, [0, 50, 500, 0, 10, 0], [1.0, 1.0, 1.0, 1.0, 1.0, ("mid", 1234)], [0.0] * 6,
          [2999, 49, 333, 1500, 9, 1234])
    x = (torch.arange(V, device="cuda") % 7).to(dtype)[None].repeat(3, 1)   # seven values, many ties each
    check(x, [1.0, 0.5, 2.0], [600, 0, 0], [1.0, ("mid", 700), 1.0], [0.0, 0.0, 0.2], [599, 650, 1200])


def test_sample_masks_nan_and_infinities():
    V = 4097
    x = logits(8, V, 4)
    ninf, inf, nan = float("-inf"), float("inf"), float("nan")
    x[0, :] = ninf                          # nothing left
    x[1, :] = ninf; x[1, 777] = -3.0        # one word left
    x[2, :] = nan                           # nothing left either
    x[3, ::2] = nan                         # NaN never wins
    x[4, 5] = inf; x[4, 4000] = inf         # two infinite logits share
    x[5, 10:] = ninf
    x[6, :] = torch.finfo(F32).min; x[6, 9] = 0.0
    x[7, :] = torch.finfo(F32).min          # all at the lowest value: equal
    rows = [1, 3, 4, 5, 6, 7]
    check(x[rows].contiguous(), [1.0] * 6, [0, 30, 0, 0, 100, 0], [1.0, ("mid", 5), 1.0, ("mid", 4), 1.0, 1.0],
          [0.0, 0.0, 0.0, 0.0, 0.0, 0.0], [0, 2, 1, 2, 3, 4000])
    ids, probs = kq.sample(x, torch.full((8,), 0.3, device="cuda"))
    torch.cuda.synchronize()
    assert ids[0] == -1 and ids[2] == -1 and probs[0] == 0 and probs[2] == 0
    assert ids[1] == 777 and probs[1] == 1 and ids[4] == 5 and ids[6] == 9


def test_sample_greedy_and_off():
    x = logits(3, 1000, 5)
    x[1, 10] = x[1, 900] = 50.0
    u = torch.tensor([0.0, 0.99, 0.5], device="cuda")
    best = x.argmax(1)
    best[1] = 10
    for t in (0.0, -1.0, float("nan")):
        ids, probs = kq.sample(x, u, temperature=torch.full((3,), t, device="cuda"))
        assert torch.equal(ids.long(), best) and torch.all(probs == 1)
    ids, _ = kq.sample(x, u, top_p=torch.zeros(3, device="cuda"))   # the first word always stays
    assert torch.equal(ids.long(), best)
    # extreme temperatures
    ids, _ = kq.sample(x, u, temperature=torch.full((3,), 1e-30, device="cuda"))
    assert ids[0] == best[0] and ids[1] == 900 and ids[2] == best[2]  # the two leaders share, u = 0.99
    ids, probs = kq.sample(x, u, temperature=torch.full((3,), 1e30, device="cuda"))
    order, _ = ranked(x[2].cpu().numpy())
    assert ids[2] == order[500]
    np.testing.assert_allclose(probs.cpu().numpy(), 1e-3, rtol=1e-5)


def test_sample_edges_of_u():
    x = logits(4, 3000, 6)
    k = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, -0.5, 1.5], device="cuda")  # outside [0, 1): the nearest word
    ids, _ = kq.sample(x, u, top_k=k)
    torch.cuda.synchronize()
    for m, r in enumerate((0, 8, 0, 8)):
        assert ids[m] == ranked(x[m].cpu().numpy())[0][r]


@pytest.mark.parametrize("M", [1, 5, 200])
def test_sample_rows_at_a_stride_and_batches(M):
    buf = logits(M, 2100, 7)
    x = buf[:, 3:2050]
    t = [0.3 + 0.01 * (m % 90) for m in range(M)]
    check(x, t, [m % 40 for m in range(M)], [1.0 if m % 3 else ("mid", m % 17) for m in range(M)],
          [0.02 * (m % 2) for m in range(M)], [m % 23 for m in range(M)])


def test_sample_frequencies():
    """Over an even grid of u the words come up in proportion to their shares."""
    x = logits(1, 500, 8)
    n = 4096
    u = (torch.arange(n, device="cuda") + 0.5) / n
    ids, probs = kq.sample(x.expand(n, 500).contiguous(), u, top_k=torch.full((n,), 30, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    order, l = ranked(x[0].cpu().numpy())
    w = weights(l[:30], 1.0)
    w /= w.sum()
    count = np.bincount(ids.cpu().numpy(), minlength=500)
    assert np.all(np.abs(count[order[:30]] - w * n) <= 1.01) and count.sum() == count[order[:30]].sum()


def test_sample_in_a_graph_and_on_another_stream():
    x = logits(7, 50000, 9)
    u = torch.rand(7, device="cuda")
    ws = kq.sample_workspace(7, 50000)
    want, wp = kq.sample(x, u, workspace=ws)
    ids, probs = torch.empty_like(want), torch.empty_like(wp)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kq.sample(x, u, workspace=ws, ids=ids, probs=probs, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(ids, want) and torch.equal(probs, wp)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kq.sample(x, u, workspace=ws, ids=ids, probs=probs)
    for _ in range(3):
        ids.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, want) and torch.equal(probs, wp)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_many_rows_some_flat(dtype):
    """More rows than the device has clusters of eight: the rows whose answer lies deep in a flat distribution, or whose
    top_k is large, are worked on apart from the others.  Twice on one workspace."""
    M, V = 160, 40001
    x = logits(M, V, 10, dtype, sd=1.0)
    x[::7] = torch.randn((len(range(0, M, 7)), V), generator=torch.Generator().manual_seed(1)).cuda().to(dtype) * 0.5
    x[3::40] = 1.0                                      # all equal
    x[5::40, 20:] = float("-inf")
    k = [[0, 20, 0, 1500, 30000][m % 5] for m in range(M)]
    p = [1.0 if m % 3 == 0 else ("mid", [3, 700, 9000][m % 3]) for m in range(M)]
    check(x, [[1.0, 0.7, 2.0][m % 3] for m in range(M)], k, p, [0.3 * (m % 11 == 0) for m in range(M)],
          [[2, 15000, 600, 39000][m % 4] for m in range(M)])


@pytest.mark.parametrize("V", [300000, 1 << 20])
def test_sample_large_vocabularies(V):
    x = logits(3, V, 11)
    check(x, [1.0, 2.5, 0.8], [0, 0, 50], [("mid", 12), 1.0, ("mid", 20)], [0.0, 0.0, 0.0], [9, 300, 5])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [6, 320])
def test_sample_total_weight_of_odd_rows(dtype, M):
    """Rows without top_k, whose every word is summed: NaN, infinities, a temperature below fp32's normal numbers, one
    logit above a flat rest, at row starts off 16 bytes."""
    V, inf = 40003, float("inf")
    base = torch.randn((6, V), generator=torch.Generator().manual_seed(12))
    base[0, ::3] = float("nan")
    base[1, [7, 39000]] = inf
    base[2, 5:] = -inf
    base[3, [11, 20000, 40002]] = 9.0
    base[4, :] = -3.0
    base[4, 33333] = 4.0
    x = base.to(dtype).cuda().repeat(M // 6 + 1, 1)[:M]
    check(x, [[1.5, 1.0, 0.7, 1e-39, 1.0, 3.0][m % 6] for m in range(M)], [0] * M,
          [[1.0, 1.0, ("mid", 3), 1.0, ("mid", 20000), 1.0][m % 6] for m in range(M)],
          [[0.0, 0.0, 0.0, 0.0, 0.0, 0.02][m % 6] for m in range(M)],
          [[9000, 1, 2, 2, [0, 15000][m // 6 % 2], 700][m % 6] for m in range(M)])
