"""kq_kv_append, kq_attn_decode and kq_sample where calls meet: one workspace for many calls, tensors on other streams, and
arguments at the ends of their types.  The 64-bit definitions and the bounds are test_gpu_cache.py's."""
import numpy as np
import pytest
import torch

from gguf_quant_weight_super_gb300 import kq, synth
from tests.gpu_util import dev, require_gpu
from tests.test_gpu_cache import BF16, F8, F32, Paged, check_attn, f64, rand_q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    require_gpu()
    from gguf_quant_weight_super_gb300 import build
    build.build()
    kq.lib()
    kq.kq_device_error(clear=True)
    yield
    assert kq.kq_device_error() == 0


def test_attn_one_workspace_for_any_calls():
    """A workspace serves calls of other batches, heads, types and row counts in turn: what one leaves in it has no
    influence on the next, down to the bits of a call on a new workspace."""
    caches = {name: Paged(lens, Hkv, D, 16, dtype, seed=i) for i, (name, lens, Hkv, D, dtype) in enumerate([
        ("batch", [700 + 41 * i for i in range(24)], 8, 128, BF16),
        ("one", [9000], 8, 128, BF16),
        ("block", [300 + 171 * i for i in range(8)], 8, 128, BF16),
        ("wide heads", [2000, 77, 1300], 4, 256, F8),
    ])}
    calls = [("batch", 1, 4, BF16), ("one", 1, 4, BF16), ("batch", 1, 4, BF16), ("block", 16, 4, BF16), ("block", 16, 4, F32),
             ("block", 16, 4, BF16), ("wide heads", 5, 4, F32), ("batch", 1, 4, F32), ("one", 16, 16, BF16), ("batch", 2, 4, BF16)]
    made = []
    for name, T, G, qt in calls:
        P = caches[name]
        made.append((P, rand_q(len(P.lens), T, G * P.cache.n_kv_heads, P.cache.head_dim, qt, T + G)))
    size = max(kq.attn_workspace(P.cache, *q.shape[:3]).numel() for P, q in made)
    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for (P, q), call in zip(made, calls):
        want = kq.attn_decode(P.cache, P.table, P.seq_lens, q, kq.attn_workspace(P.cache, *q.shape[:3]))
        got = torch.full_like(q, float("nan"))
        kq.attn_decode(P.cache, P.table, P.seq_lens, q, shared, out=got)
        torch.cuda.synchronize()
        assert torch.equal(got, want), call


@pytest.mark.parametrize("qt", [BF16, F32])
@pytest.mark.parametrize("D,T,G", [(64, 1, 1), (128, 1, 8), (128, 8, 4), (256, 1, 2), (256, 3, 4)])
@pytest.mark.parametrize("n,B", [(200, 1), (3000, 1), (300, 600)])
def test_attn_8bit_small_weights_beside_a_peak(qt, D, T, G, n, B):
    """One score 16 to 18.5 above the rest, its value 0: the result is made of weights below 2^-23 of the largest.  The
    bound of test_gpu_cache.py, and 2^-40 of the largest weight for each position: 2^15 times a weight enters as two fp16
    parts, whose steps end at 2^-24."""
    P = Paged([n], 1, D, 64, F8, seed=D + n)
    g = torch.Generator().manual_seed(n)
    k, v = torch.zeros(P.k.shape), torch.zeros(P.v.shape)
    k[..., 0] = 1.5 + 2.5 * torch.rand(P.k.shape[:-1], generator=g)
    v[:] = 0.5 + torch.rand(P.v.shape, generator=g)
    first = int(P.table[0, 0])
    k[first, 0, :, 0], v[first, 0] = 20.0, 0.0
    P.k.copy_((k / P.k_scale).to(F8)), P.v.copy_((v / P.v_scale).to(F8))
    q = torch.zeros((B, T, G, D), dtype=qt, device="cuda")
    q[..., 0] = 1.0
    table, lens = P.table.expand(B, -1).contiguous(), P.seq_lens.expand(B).contiguous()  # all read the same pages
    out = kq.attn_decode(P.cache, table, lens, q, kq.attn_workspace(P.cache, B, T, G), scale=1.0)
    torch.cuda.synchronize()
    kk, vv = (x[:, 0] for x in P.dense(0))
    for t in range(T):
        m = n - T + t + 1
        s = kk[:m, 0]
        p = np.exp(s - s.max())
        ref, sv, lost = p @ vv[:m] / p.sum(), p @ np.abs(vv[:m]) / p.sum(), 2.0 ** -40 * np.abs(vv[:m]).sum(0) / p.sum()
        part, rnd = (2.0 ** -16, 2.0 ** -8) if qt == BF16 else (2.0 ** -20, 2.0 ** -24)
        d = 2 * (D + 8) * 2.0 ** -23 * np.abs(kk[:m]).max() + 2.0 ** -20 + part + (n / 8 + 128) * 2.0 ** -23
        tol = (d * sv + lost) * (1 + rnd) + rnd * np.abs(ref)
        err = np.abs(f64(out.float())[:, t] - ref)
        assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("T,G", [(1, 4), (16, 4)])
def test_attn_longest_lengths(T, G):
    """Lengths at the end of 32 bits, all pages of a sequence being one: the last positions as at length 2048, and a
    length past the limit is recorded and keeps the other sequence as it is."""
    P = Paged([1024, 500], 1, 64, 1024, BF16, seed=50)
    q = rand_q(2, T, G, 64, BF16, 51)
    ws = kq.attn_workspace(P.cache, 2, T, G)
    table = P.table[:, :1].expand(2, 1 << 21).contiguous()

    def call(n):
        lens = torch.tensor([n, 500], dtype=torch.int32, device="cuda")
        out = kq.attn_decode(P.cache, table, lens, q, ws, window=100)
        torch.cuda.synchronize()
        return out

    want = call(2048)
    assert torch.equal(call(2 ** 31 - 4096), want) and kq.kq_device_error() == 0
    got = call(2 ** 31 - 1)
    assert kq.kq_device_error(clear=True) == 4
    assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,G,Hkv", [(8, 4, 2), (16, 4, 2), (16, 1, 32), (3, 2, 1)])
def test_attn_largest_windows_are_none(T, G, Hkv):
    """Windows of the table's positions and more, up to the largest, cut nothing, beside padding tokens too."""
    P = Paged([1, 500, 1, 1, 37], Hkv, 64, 16, BF16, seed=52)
    q = rand_q(5, T, G * Hkv, 64, BF16, 53)
    ws = kq.attn_workspace(P.cache, 5, T, G * Hkv)
    want = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws)
    room = P.table.shape[1] * 16
    for window in (2 ** 31 - 1, 2 ** 31 - 8, 1 << 30, room + 1, room, room - 1):
        out = torch.full_like(q, float("nan"))
        kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out, want), window


@pytest.mark.parametrize("rot", [0, 64])
def test_append_negative_lengths_are_padding(rot):
    """A length below 0, down to the lowest, is a sequence of padding tokens: zeros out, nothing stored, no error."""
    P = Paged([0, 9, 0], 2, 64, 16, BF16, seed=54, fill="zero")
    lens = torch.tensor([-2 ** 31, 9, -1], dtype=torch.int32, device="cuda")
    q, kv = rand_q(3, 3, 4, 64, BF16, 55), rand_q(3, 3, 2, 64, BF16, 56)
    out = kq.kv_append(P.cache, P.table, lens, q, kv, kv, kq.RopeNorm(kq.rope_table(20, 64)) if rot else kq.RopeNorm())
    torch.cuda.synchronize()
    assert kq.kq_device_error(clear=True) == 0
    assert torch.all(out[0] == 0) and torch.all(out[1] != 0) and torch.all(out[2] == 0)
    stored = (P.k.nan_to_num(0.0) != 0).any(-1).any(-1)
    assert int(stored.sum()) == 3 and torch.all(stored[int(P.table[1, 0]), 6:9])


@pytest.mark.parametrize("handle", [False, True])
def test_tensors_of_a_call_on_another_stream(handle):
    """What a call makes itself (outputs, the sampler's workspace) is ordered with the stream it is given: it is neither a
    block that pending work of the current stream still writes, nor filled on the current stream."""
    P = Paged([300, 40], 2, 128, 16, BF16, seed=57)
    q, kv = rand_q(2, 1, 8, 128, BF16, 58), rand_q(2, 1, 2, 128, BF16, 59)
    ws = kq.attn_workspace(P.cache, 2, 1, 8)
    side = torch.cuda.Stream()
    x, u = torch.randn(40, 40000, device="cuda"), torch.full((40,), 0.5, device="cuda")  # flat: half of them go to the tail
    k = torch.tensor([5, 3000] * 20, dtype=torch.int32, device="cuda")
    route = torch.randn(3, 16, device="cuda")

    def calls(stream):
        yield lambda: [kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, stream=stream)]
        yield lambda: [kq.kv_append(P.cache, P.table, P.seq_lens, q, kv, kv, kq.RopeNorm(), stream=stream)]
        yield lambda: list(kq.sample(x, u, top_k=k, stream=stream))
        yield lambda: list(kq.moe_route(route, 2, stream=stream))

    for plain, there in zip(calls(None), calls(side.cuda_stream if handle else side)):
        want = plain()
        sizes = [t.shape for t in want] + [(2048,)]  # the sampler's workspace is of a few KB
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        for shape in sizes:  # written after the sleep, their blocks are free for the current stream at once
            torch.empty(shape, device="cuda").fill_(1e9)
        got = there()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    a = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, stream=0)  # the default stream's handle
    b = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_chain_planned_on_another_stream():
    """A chain's workspace holds its plan: pending work of the current stream does not write over it."""
    N, K = 64, 512
    W = dev(synth.gen_matrix(synth.Q4_K, N, K, synth.rng(600)))
    x, y, want = torch.randn(1, K, device="cuda"), torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    op = dict(type=synth.Q4_K, x_dtype=kq.KQ_F32, W=W, x=x, N=N, K=K)
    kq.Chain([dict(op, y=want)]).run()
    size = kq.kq_chain_workspace_size([dict(op, y=y)]) + 256
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)
    torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0)
    chain = kq.Chain([dict(op, y=y)], stream=side)
    torch.cuda.synchronize()  # whatever was pending has been written
    chain.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F8])
@pytest.mark.parametrize("qt", [kq.KQ_BF16, kq.KQ_F32])
def test_attn_ranges_are_all_resident(D, dtype, qt):
    """The line of tiles is cut for CTAs that run at the same time: the device holds as many as the kernel is laid out for,
    up to 256 sequences; a large batch's index leaves room for one at least."""
    c = kq.KVCache(*(torch.zeros((1, 16, 1, D), device="cuda").to(dtype) for _ in range(2)))
    for rows in (1, 8, 9, 16, 17, 32, 128, 256):
        T, G = max(1, rows // 16), min(rows, 16)
        if T * G != rows:
            T, G = rows, 1
        if T > 16:
            T, G = 16, 2
        planned, resident = kq.kq_selftest_attn_ctas(c._ref, 1, T, qt, G)
        assert planned == resident >= 1, (rows, planned, resident)
        at_256 = kq.kq_selftest_attn_ctas(c._ref, 256, T, qt, G)  # of more than 16 rows maybe the other kernel's
        assert at_256[0] == at_256[1] and (rows > 16 or at_256[0] == planned), (rows, at_256)
        assert kq.kq_selftest_attn_ctas(c._ref, 4096, T, qt, G)[1] >= 1
        if rows <= 8 and dtype == BF16 and qt == kq.KQ_BF16 and D <= 128:
            assert planned == 3


def test_attn_large_batch_with_fewer_ranges():
    """4096 sequences: the index takes a CTA's place on each SM."""
    lens = [(i * 37) % 100 for i in range(4096)]
    P = Paged([99], 1, 128, 16, BF16, seed=60)
    q = rand_q(4096, 1, 2, 128, BF16, 61)
    table = P.table.expand(4096, -1).contiguous()
    out = kq.attn_decode(P.cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, kq.attn_workspace(P.cache, 4096, 1, 2))
    few = list(range(0, 4096, 256))
    want = kq.attn_decode(P.cache, table[few].contiguous(), torch.tensor([lens[i] for i in few], dtype=torch.int32, device="cuda"),
                          q[few].contiguous(), kq.attn_workspace(P.cache, len(few), 1, 2))
    torch.cuda.synchronize()
    # the same sums in another order and one rounding to bf16
    assert torch.all((out[few].double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -14)
    assert torch.all(out[lens.index(0)] == 0)


@pytest.mark.parametrize("qt", [BF16, F32])
@pytest.mark.parametrize("D,Hkv,G", [(64, 2, 1), (128, 2, 4), (256, 1, 2)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_attn_8bit_nan_in_unseen_positions(qt, D, Hkv, G, what):
    """As test_attn_unseen_positions_do_not_matter, in an e4m3 cache, whose only special value is NaN."""
    T, n, window = 8, 200, 64
    P = Paged([n, 64], Hkv, D, 16, F8, seed=62)
    q = rand_q(2, T, G * Hkv, D, qt, 63)
    ws = kq.attn_workspace(P.cache, 2, T, G * Hkv)
    clean = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window)
    for pos in (n - 3, n - T - window + 3):  # seen by tokens t >= 5; by tokens t <= 2
        (P.k if what == "k" else P.v).view(torch.uint8)[int(P.table[0, pos // 16]), pos % 16, 0, 5] = 0x7F
    got = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window)
    torch.cuda.synchronize()
    for t in range(T):
        if 2 < t < 5:
            assert torch.equal(got[0, t], clean[0, t]), t
            continue
        assert torch.equal(got[0, t, G:], clean[0, t, G:]), t
        nan = torch.isnan(got[0, t, :G])
        assert torch.all(nan if what == "k" else nan[:, 5]), t
        if what == "v":
            rest = [d for d in range(D) if d != 5]
            assert torch.equal(got[0, t, :G][:, rest], clean[0, t, :G][:, rest]), t
    assert torch.equal(got[1], clean[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,Hkv,G", [(2, 16, 1, 2), (3, 5, 2, 4), (33, 8, 1, 4), (5, 10, 2, 4), (7, 11, 1, 3), (6, 16, 4, 4),
                                       (3, 16, 4, 4), (12, 16, 2, 8), (2, 16, 2, 8), (7, 15, 4, 9), (6, 16, 4, 16), (1, 16, 2, 16)])
def test_attn_blocks_of_few_and_many_heads(D, B, T, Hkv, G):
    """Blocks of more than 16 rows, on both sides of the choice between the kernels, with a window and without."""
    lens = [(517, 100, 16, 0, 3, 64, 1030)[i % 7] for i in range(B)]
    P = Paged(lens, Hkv, D, 32, BF16, seed=T * G + B)
    q = rand_q(B, T, Hkv * G, D, BF16, 64)
    check_attn(P, q)
    check_attn(P, q, cap=20.0, window=70)


@pytest.mark.parametrize("what", ["v_nan", "k_nan", "v_inf"])
@pytest.mark.parametrize("T,G", [(8, 8), (16, 8), (16, 16)])
def test_attn_unseen_positions_of_many_rows(what, T, G):
    """As test_attn_unseen_positions_do_not_matter, for blocks of 64 rows and more of many heads."""
    n, window, Hkv, B = 200, 64, 8, 4
    P = Paged([n, 64, 300, 17], Hkv, 128, 16, BF16, seed=65)
    q = rand_q(B, T, G * Hkv, 128, BF16, 66)
    ws = kq.attn_workspace(P.cache, B, T, G * Hkv)
    clean = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window)
    bad = float("inf") if what == "v_inf" else float("nan")
    late, early = n - 3, n - T - window + 3  # seen by tokens from T - 3 on; by tokens up to 2
    for pos in (late, early):
        (P.k if what == "k_nan" else P.v)[int(P.table[0, pos // 16]), pos % 16, 0, 3] = bad
    got = kq.attn_decode(P.cache, P.table, P.seq_lens, q, ws, window=window)
    torch.cuda.synchronize()
    rest = [d for d in range(128) if d != 3]
    for t in range(T):
        assert torch.equal(got[0, t, G:], clean[0, t, G:]), t
        mine = got[0, t, :G].float()
        if 2 < t < T - 3:
            assert torch.equal(got[0, t, :G], clean[0, t, :G]), t
        elif what == "k_nan":
            assert torch.all(torch.isnan(mine)), t
        else:
            assert torch.all(torch.isnan(mine[:, 3]) if what == "v_nan" else torch.isinf(mine[:, 3])), t
            assert torch.equal(mine[:, rest], clean[0, t, :G].float()[:, rest]), t
    assert torch.equal(got[1:], clean[1:])
