"""The decode step's operators around the quantized products, in their plain
form and as calls of the library: what they cost and how exact they are.

Three operators: kv_append (per-head norms of q and k, rotary positions, k and
v written into a paged cache), attn_decode (attention of the newest 1..16
tokens of each sequence over that cache) and sample (temperature, top-k,
top-p, min-p from given uniform numbers)."""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # One chat, a short history: a step's attention is all latency.  The
        # head layout of the 4B-class decoder (32 heads on 8 of 128).
        dict(name="attn_one_short", op="attn", B=1, T=1, Hkv=8, G=4, D=128, L=1000, spread=0.0, page=16,
             q="bf16", cache="bf16", window=0, cap=0.0, lens=1),
        # A serving batch whose histories differ a lot, empty slots among them.
        dict(name="attn_ragged_batch", op="attn", B=24, T=1, Hkv=8, G=4, D=128, L=9001, spread=1.0, page=32,
             q="bf16", cache="bf16", window=0, cap=0.0, lens=2),
        # Four long documents.
        dict(name="attn_long", op="attn", B=4, T=1, Hkv=8, G=4, D=128, L=131071, spread=0.1, page=64,
             q="bf16", cache="bf16", window=0, cap=0.0, lens=3),
        # Speculative verification: 16 drafted tokens of each of 8 sequences at once.
        dict(name="attn_verify", op="attn", B=8, T=16, Hkv=8, G=4, D=128, L=6007, spread=0.5, page=16,
             q="bf16", cache="bf16", window=0, cap=0.0, lens=4),
        # A local layer of wide heads: window, capped scores, an 8-bit cache, fp32 queries.
        dict(name="attn_window_cap_fp8", op="attn", B=16, T=1, Hkv=4, G=2, D=256, L=20011, spread=0.6, page=64,
             q="f32", cache="fp8", window=4096, cap=50.0, lens=5),
        # One new token: fp32 q, k, v as the products leave them.
        dict(name="append_one", op="append", B=1, T=1, Hq=32, Hkv=8, D=128, L=1000, page=16, x="f32", q="bf16",
             cache="bf16", norm=True, off=0.0, rot=128, inter=False, fused=False, lens=6),
        # A verify block of 16 sequences, one fused bf16 qkv buffer, no norms, interleaved pairs on half of the head.
        dict(name="append_verify", op="append", B=16, T=8, Hq=32, Hkv=8, D=128, L=5003, page=32, x="bf16", q="bf16",
             cache="bf16", norm=False, off=0.0, rot=64, inter=True, fused=True, lens=7),
        # Prompts on their way into an 8-bit cache, zero-centred norm weights.
        dict(name="append_prompt", op="append", B=4, T=2047, Hq=16, Hkv=4, D=256, L=2047, page=64, x="f32", q="bf16",
             cache="fp8", norm=True, off=1.0, rot=256, inter=False, fused=False, lens=8),
        # One token of a 151936-word vocabulary, the usual chat settings.
        dict(name="sample_one", op="sample", M=1, V=151936, x="f32", temp=0.7, k=20, p=0.8, minp=0.0, masked=0),
        # A verify block's 16 rows of a 262144-word vocabulary: nucleus and min-p without top-k.
        dict(name="sample_verify", op="sample", M=16, V=262144, x="f32", temp=1.0, k=0, p=0.95, minp=0.02, masked=4),
        # A large batch of bf16 logits (many equal), a different setting in each row, some rows behind a grammar's mask.
        dict(name="sample_batch", op="sample", M=256, V=151936, x="bf16", temp=-1.0, k=-1, p=-1.0, minp=-1.0, masked=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "sample"])
    if op == "attn":
        T = rng.choice([1, 1, 1, rng.randint(2, 4), rng.randint(5, 16)])
        D = rng.choice([64, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        B = _log(rng, 1, 64)
        room = 4 * 131071 * 8 * 128 // 2          # cache values of one side, half of the longest listed case's
        room = min(room, room * 64 // (T * G))     # and the scores' cost
        L = _log(rng, 1, max(1, min(150000, room // (B * Hkv * D))))
        return dict(op="attn", B=B, T=T, Hkv=Hkv, G=G, D=D, L=L, spread=rng.choice([0.0, 0.5, 1.0]),
                    page=rng.choice([8, 16, 32, 64, 128]), q=rng.choice(["bf16", "bf16", "f32"]),
                    cache=rng.choice(["bf16", "bf16", "fp8"]), window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), lens=rng.randrange(1 << 20))
    if op == "append":
        D, Hkv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        B = _log(rng, 1, 128)
        T = _log(rng, 1, max(1, 4 * 2047 * 24 * 256 // (B * (Hq + 2 * Hkv) * D)))
        T = min(T, 4096)
        return dict(op="append", B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, L=T + _log(rng, 1, 20000),
                    page=rng.choice([8, 16, 32, 64, 128]), x=rng.choice(["f32", "bf16"]),
                    q=rng.choice(["bf16", "bf16", "f32"]), cache=rng.choice(["bf16", "bf16", "fp8"]),
                    norm=rng.random() < 0.6, off=rng.choice([0.0, 1.0]), rot=rng.choice([D, D, D // 2]),
                    inter=rng.random() < 0.4, fused=rng.random() < 0.5, lens=rng.randrange(1 << 20))
    V = _log(rng, 1000, 262144)
    return dict(op="sample", M=_log(rng, 1, max(1, 256 * 151936 // V)) if V > 20000 else _log(rng, 1, 512), V=V,
                x=rng.choice(["f32", "bf16"]), temp=rng.choice([0.6, 1.0, -1.0]), k=rng.choice([0, 1, 20, 64, 1000, -1]),
                p=rng.choice([1.0, 0.9, 0.95, -1.0]), minp=rng.choice([0.0, 0.05, -1.0]), masked=rng.choice([0, 0, 4]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


def _lengths(case):
    """The sequences' lengths, the new tokens included: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    if case["op"] == "append":
        return [r.randint(case["T"], case["L"]) for _ in range(case["B"])]
    lens = [max(0, int(case["L"] * (1.0 - case["spread"] * r.random()))) for _ in range(case["B"])]
    if case["spread"] == 1.0 and case["B"] >= 4:
        lens[r.randrange(case["B"])] = 0  # an empty slot of the batch
        lens[r.randrange(case["B"])] = 1
    return lens


def _randn(shape, dtype, g, mul=1.0):
    if dtype == torch.float8_e4m3fn:
        out = torch.empty(shape, dtype=dtype, device="cuda")
        flat, n = out.view(-1), out.numel()
        for i in range(0, n, 1 << 27):
            j = min(n, i + (1 << 27))
            flat[i:j] = (torch.randn(j - i, device="cuda", generator=g) * mul).to(dtype)
        return out
    x = torch.randn(shape, dtype=dtype, device="cuda", generator=g)
    return x if mul == 1.0 else x.mul_(mul)


def _rope_table(n, rot, base=1000000.0):
    """cos | sin of each position's angles, made in 64 bits once."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _paged(case, lens, g):
    """A pool of pages in which the sequences' pages lie in any order, and the table of each sequence's pages."""
    P = case["page"]
    used = [-(-n // P) for n in lens]
    if case["op"] == "append":  # only the pages that the new tokens go to are present
        T = case["T"]
        first = [(n - T) // P for n in lens]
        need = [u - f for u, f in zip(used, first)]
    else:
        first, need = [0] * len(lens), used
    width, total = max(1, max(used)), sum(need)
    n_pages = total + 3
    ids = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), width), 0, dtype=torch.int32, device="cuda")
    at = 0
    for b, (f, m) in enumerate(zip(first, need)):
        table[b, f:f + m] = ids[at:at + m]
        at += m
    return n_pages, table


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    s = dict(case)
    if case["op"] == "sample":
        return _prepare_sample(s, case, g)
    lens = _lengths(case)
    B, T, Hkv, D, P = case["B"], case["T"], case["Hkv"], case["D"], case["page"]
    n_pages, s["table"] = _paged(case, lens, g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ct = _TYPES[case["cache"]]
    s["k_scale"], s["v_scale"] = (0.02, 0.015) if case["cache"] == "fp8" else (1.0, 1.0)
    if case["op"] == "attn":
        Hq = Hkv * case["G"]
        # slots past a sequence's end keep what an earlier user left: any values
        s["k"] = _randn((n_pages, P, Hkv, D), ct, g, 1.0 / s["k_scale"] if ct == torch.float8_e4m3fn else 1.0)
        s["v"] = _randn((n_pages, P, Hkv, D), ct, g, 1.0 / s["v_scale"] if ct == torch.float8_e4m3fn else 1.0)
        s["q"] = _randn((B, T, Hq, D), _TYPES[case["q"]], g, 2.0)  # peaked scores
        s["scale"] = D ** -0.5
        s["out"] = torch.empty_like(s["q"])
    else:
        Hq, xt = case["Hq"], _TYPES[case["x"]]
        s["k"] = torch.zeros((n_pages, P, Hkv, D), dtype=ct, device="cuda")
        s["v"] = torch.zeros((n_pages, P, Hkv, D), dtype=ct, device="cuda")
        if case["fused"]:
            x = _randn((B, T, Hq + 2 * Hkv, D), xt, g, 1.5)
            s["xq"], s["xk"], s["xv"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        else:
            s["xq"], s["xk"], s["xv"] = (_randn((B, T, h, D), xt, g, 1.5) for h in (Hq, Hkv, Hkv))
        s["eps"] = 1e-6
        centre = 1.0 - case["off"]
        s["wq"], s["wk"] = ((centre + 0.2 * torch.randn(D, device="cuda", generator=g) for _ in range(2))
                            if case["norm"] else (None, None))
        s["table_cs"] = _rope_table(case["L"], case["rot"])
        s["q"] = torch.empty((B, T, Hq, D), dtype=_TYPES[case["q"]], device="cuda")
    if own:  # the handles that a serving program makes once
        from gguf_quant_weight_super_gb300 import kq
        s["cache_h"] = kq.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "attn":
            s["ws"] = kq.attn_workspace(s["cache_h"], B, T, Hq)
        else:
            s["rope_h"] = kq.RopeNorm(s["table_cs"], interleaved=case["inter"], q_norm=s["wq"], k_norm=s["wk"],
                                      eps=s["eps"], norm_offset=case["off"])
    return s


def _prepare_sample(s, case, g):
    M, V = case["M"], case["V"]
    # a wide bulk and a few dozen likely words in each row, as a language model's head gives
    x = torch.randn((M, V), device="cuda", generator=g) * 2.0
    top = torch.randint(0, V, (M, 48), device="cuda", generator=g)
    x.scatter_add_(1, top, 4.0 + 12.0 * torch.rand((M, 48), device="cuda", generator=g))
    if case["masked"]:  # a grammar leaves a few words of every `masked`-th row
        rows = torch.arange(M, device="cuda") % case["masked"] == 0
        off = torch.rand((M, V), device="cuda", generator=g) < 0.995
        x.masked_fill_(off & rows[:, None], float("-inf"))
        x[:, 0] = torch.where(rows, x[:, 1:].amax(1).clamp(min=0.0), x[:, 0])
    s["x"] = x.to(_TYPES[case["x"]])
    del x

    def par(value, choices, dtype):
        c = torch.tensor(choices, dtype=dtype, device="cuda")
        pick = torch.randint(0, len(choices), (M,), device="cuda", generator=g)
        return c[pick] if value < 0 else torch.full((M,), value, dtype=dtype, device="cuda")

    s["temp"] = par(case["temp"], [0.0, 0.3, 0.6, 0.8, 1.0, 1.3], torch.float32)
    s["top_k"] = par(case["k"], [0, 1, 5, 20, 40, 100, 1000], torch.int32)
    s["top_p"] = par(case["p"], [0.5, 0.8, 0.9, 0.95, 1.0], torch.float32)
    s["min_p"] = par(case["minp"], [0.0, 0.0, 0.02, 0.1], torch.float32)
    # The uniform numbers.  One that falls within 1e-5 of the edge between two
    # words has no answer in 32 bits and is drawn again.
    u = torch.rand((16, M), device="cuda", generator=g)
    edges = _edges64(s)
    s["u"] = (0.5 * edges[:, 0]).float()
    good = torch.zeros(M, dtype=torch.bool, device="cuda")
    for i in range(16):
        at = torch.searchsorted(edges, u[i].double()[:, None])
        lo = edges.gather(1, (at - 1).clamp(min=0))[:, 0]
        hi = edges.gather(1, at.clamp(max=edges.shape[1] - 1))[:, 0]
        ud = u[i].double()
        ok = (((ud - lo).abs() > 1e-5) | (at[:, 0] == 0)) & ((hi - ud).abs() > 1e-5) & (ud < hi)
        s["u"] = torch.where(~good & ok, u[i], s["u"])
        good |= ok
    s["ids"] = torch.empty(M, dtype=torch.int32, device="cuda")
    s["probs"] = torch.empty(M, dtype=torch.float32, device="cuda")
    if own:
        from gguf_quant_weight_super_gb300 import kq
        s["ws"] = kq.sample_workspace(M, V)
    return s


def _edges64(s):
    """Each row's running share of the kept probability in descending order of the logits, in 64 bits."""
    M, V = s["x"].shape
    out = torch.empty((M, min(V, 1 << 14)), dtype=torch.float64, device="cuda")  # later edges: nearer than 1e-5 anyway
    for i in range(0, M, 32):
        x = s["x"][i:i + 32].double().sort(1, descending=True).values
        t = s["temp"][i:i + 32].double()[:, None]
        w = torch.where(t > 0, ((x - x[:, :1]) / t.clamp(min=1e-30)).exp(), 0.0)
        w[:, 0] = 1.0
        k = s["top_k"][i:i + 32].long()[:, None]
        w *= (torch.arange(V, device="cuda") < torch.where(k > 0, k, V))
        c = w.cumsum(1)
        p = s["top_p"][i:i + 32].double()[:, None]
        keep = ((c - w) < p * c[:, -1:]) | (p >= 1)
        keep &= w >= s["min_p"][i:i + 32].double()[:, None]
        keep[:, 0] = True
        c = (w * keep).cumsum(1)
        out[i:i + 32] = (c / c[:, -1:])[:, :out.shape[1]]
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from gguf_quant_weight_super_gb300 import kq
    if s["op"] == "attn":
        return kq.attn_decode(s["cache_h"], s["table"], s["lens"], s["q"], s["ws"], scale=s["scale"], softcap=s["cap"],
                              window=s["window"], out=s["out"])
    if s["op"] == "append":
        kq.kv_append(s["cache_h"], s["table"], s["lens"], s["xq"], s["xk"], s["xv"], s["rope_h"], q_out=s["q"])
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    ids, probs = kq.sample(s["x"], s["u"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                           min_p=s["min_p"], workspace=s["ws"], ids=s["ids"], probs=s["probs"])
    return {"ids": ids, "probs": probs}


def _run_plain(s):
    return {"attn": _plain_attn, "append": _plain_append, "sample": _plain_sample}[s["op"]](s)


def _plain_attn(s):
    B, T, Hq, D = s["q"].shape
    Hkv = s["Hkv"]
    L = s["table"].shape[1] * s["page"]
    k = s["k"][s["table"]].float().view(B, L, Hkv, D) * s["k_scale"]
    v = s["v"][s["table"]].float().view(B, L, Hkv, D) * s["v_scale"]
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, T, Hq // Hkv, L) * s["scale"]
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    j = torch.arange(L, device="cuda")
    at = s["lens"][:, None] - T + torch.arange(T, device="cuda")     # each new token's position
    see = j <= at[:, :, None]
    if s["window"]:
        see = see & (j > at[:, :, None] - s["window"])
    x = x.masked_fill(~see[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total == 0, 1.0, total)
    v = torch.where((j < s["lens"][:, None])[:, :, None, None], v, 0.0)
    o = torch.matmul(w.view(B, Hkv, -1, L), v.permute(0, 2, 1, 3)).view(B, Hkv, T, -1, D)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(s["q"].dtype)


def _plain_norm(x, w, off, eps):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (w + off)


def _plain_rotate(x, c, sn, rot, inter):
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    y1, y2 = a * c - b * sn, b * c + a * sn
    y = torch.stack([y1, y2], -1).flatten(-2) if inter else torch.cat([y1, y2], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_store(pool, x, page, slot, scale):
    x = x / scale
    pool[page, slot] = x.clamp(-448.0, 448.0).to(pool.dtype) if pool.dtype == torch.float8_e4m3fn else x.to(pool.dtype)


def _plain_append(s):
    T, rot, P = s["T"], s["rot"], s["page"]
    at = s["lens"][:, None].long() - T + torch.arange(T, device="cuda")
    cs = s["table_cs"][at]
    c, sn = cs[:, :, None, :rot // 2], cs[:, :, None, rot // 2:]
    q = _plain_rotate(_plain_norm(s["xq"].float(), s["wq"], s["off"], s["eps"]), c, sn, rot, s["inter"])
    k = _plain_rotate(_plain_norm(s["xk"].float(), s["wk"], s["off"], s["eps"]), c, sn, rot, s["inter"])
    page, slot = s["table"].long().gather(1, at // P), at % P
    _plain_store(s["k"], k, page, slot, s["k_scale"])
    _plain_store(s["v"], s["xv"].float(), page, slot, s["v_scale"])
    return {"q": q.to(s["q"].dtype), "k": s["k"], "v": s["v"]}


def _plain_sample(s):
    x = s["x"].float()
    V = x.shape[1]
    x = torch.where(torch.isnan(x), float("-inf"), x)
    x, idx = torch.sort(x, dim=1, descending=True, stable=True)
    t = s["temp"][:, None]
    z = torch.where(x == x[:, :1], 0.0, (x - x[:, :1]) / torch.where(t > 0, t, 1.0))
    r = torch.arange(V, device="cuda")
    k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None]
    k = torch.where(t > 0, k, 1)
    w = torch.exp(z) * (r < k)
    c = torch.cumsum(w, 1)
    p = s["top_p"][:, None]
    keep = (((c - w) < p * c[:, -1:]) | (p >= 1)) & (w >= s["min_p"][:, None])
    w = torch.where(keep | (r == 0), w, 0.0)
    c = torch.cumsum(w, 1)
    total = c[:, -1:]
    at = (c <= s["u"][:, None] * total).sum(1, keepdim=True)
    at = torch.minimum(at, (w > 0).sum(1, keepdim=True) - 1)
    none = x[:, :1] == float("-inf")
    ids = torch.where(none, -1, idx.gather(1, at))[:, 0].to(torch.int32)
    probs = torch.where(none, 0.0, w.gather(1, at) / total)[:, 0]
    return {"ids": ids, "probs": probs}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        return {"bytes": M * V * _BYTES[case["x"]] + M * 28, "flops": 4.0 * M * V}
    lens, T, Hkv, D = _lengths(case), case["T"], case["Hkv"], case["D"]
    if case["op"] == "append":
        n, Hq = case["B"] * T, case["Hq"]
        return {"bytes": n * (Hq + 2 * Hkv) * D * _BYTES[case["x"]] + n * case["rot"] * 4 + n * Hq * D * _BYTES[case["q"]]
                + 2 * n * Hkv * D * _BYTES[case["cache"]], "flops": 10.0 * n * (Hq + Hkv) * D}
    Hq, W = Hkv * case["G"], case["window"]
    union, pairs = 0, 0  # keys that some new token sees; (token, key) pairs
    for n in lens:
        first = max(0, n - T)
        union += n - (max(0, first - W + 1) if W else 0)
        pairs += sum(min(p + 1, W) if W else p + 1 for p in range(first, n))
    return {"bytes": 2 * union * Hkv * D * _BYTES[case["cache"]] + 2 * case["B"] * T * Hq * D * _BYTES[case["q"]]
            + 4 * sum(-(-n // case["page"]) for n in lens), "flops": 4.0 * pairs * Hq * D}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "sample": _exact_sample}[case["op"]](case, s)


def _exact_attn(case, s):
    B, T, Hq, D = s["q"].shape
    Hkv, P, G = case["Hkv"], case["page"], case["G"]
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        lo = max(0, n - T - case["window"]) if case["window"] else 0
        pages = s["table"][b, :-(-n // P)].long()
        j = torch.arange(lo, n, device="cuda")
        for h in range(Hkv):
            k = s["k"][:, :, h][pages[j // P], j % P].double() * s["k_scale"]
            v = s["v"][:, :, h][pages[j // P], j % P].double() * s["v_scale"]
            for t in range(T):
                pos = n - T + t
                if pos < 0:
                    continue
                first = max(lo, pos - case["window"] + 1) if case["window"] else 0
                a, e = first - lo, pos + 1 - lo
                x = s["q"][b, t, h * G:(h + 1) * G].double() @ k[a:e].T * s["scale"]
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                out[b, t, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v[a:e]
    return out


def _exact_append(case, s):
    T, P, rot, D = case["T"], case["page"], case["rot"], case["D"]
    half = rot // 2
    first = torch.arange(half, device="cuda") * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else half)
    k_pool, v_pool = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    qs = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        pos = torch.arange(n - T, n, device="cuda")
        cos, sin = s["table_cs"][pos, :half].double()[:, None], s["table_cs"][pos, half:].double()[:, None]
        turned = []
        for x, w in ((s["xq"][b], s["wq"]), (s["xk"][b], s["wk"])):
            x = x.double()
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * (w.double() + case["off"])
            y = x.clone()
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., second] * cos + x[..., first] * sin
            turned.append(y)
        qs[b] = turned[0]
        where = (s["table"][b].long()[pos // P], pos % P)
        k_pool[where] = turned[1] / s["k_scale"]
        v_pool[where] = s["xv"][b].double() / s["v_scale"]
    if case["cache"] == "fp8":
        k_pool.clamp_(-448, 448), v_pool.clamp_(-448, 448)
    return {"q": qs, "k": k_pool, "v": v_pool}


def _exact_sample(case, s):
    """By the definition, row by row: the words in order of their logits, cut three times, then walked."""
    ids, probs = [], []
    for m in range(case["M"]):
        x, idx = s["x"][m].double().sort(descending=True, stable=True)
        t, k, p, mp, u = (s[n][m].item() for n in ("temp", "top_k", "top_p", "min_p", "u"))
        n = 1 if t == 0 else min(case["V"], k) if k > 0 else case["V"]
        w = ((x[:n] - x[0]) / (t if t > 0 else 1.0)).exp()
        c = w.cumsum(0)
        if p < 1:
            n = min(n, max(1, int((c - w < p * c[-1]).sum())))
        n = min(n, max(1, int((w >= mp).sum())))
        at = min(n - 1, int((c[:n] <= u * c[n - 1]).sum()))
        ids.append(int(idx[at]))
        probs.append(float(w[at] / c[n - 1]))
    return {"ids": torch.tensor(ids, dtype=torch.int32), "probs": torch.tensor(probs, dtype=torch.float64)}
