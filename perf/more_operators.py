"""Operators for trees of drafted tokens and for caches of latent vectors, in
their plain form and as calls of the library: what they cost and how exact
they are.

  append_tree    kv_append of drafted tokens that form a tree (position != slot)
  attn_tree      attention of such a tree over the paged cache
  accept         the walk along the accepted branch, and its keys and values
                 moved together in every layer's cache
  latent_append  norm, rotation and write of one latent vector per token, and
                 the queries that go with it
  latent_attn    attention whose keys and values are those vectors (absorbed
                 form), of chains and trees

A tree is a 64-bit mask per drafted token: bit u says that it sees drafted
token u (its ancestors and itself); a mask of 0 is padding."""
import math
import random

import torch

own = False

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # One chat, a drafted tree of 16 nodes over a short history: all latency.  32 heads on 8 of 128.
        dict(name="attn_tree_one", op="attn_tree", B=1, T=16, Hkv=8, G=4, D=128, L=1000, spread=0.0, page=16, q="bf16",
             cache="bf16", window=0, cap=0.0, lens=11),
        # A batch of sequences with trees of up to 61 nodes, some smaller, one slot empty.
        dict(name="attn_tree_batch", op="attn_tree", B=8, T=61, Hkv=8, G=4, D=128, L=6007, spread=1.0, page=16, q="bf16",
             cache="bf16", window=0, cap=0.0, lens=12),
        # A local layer of wide heads: window, capped scores, an 8-bit cache, fp32 queries.
        dict(name="attn_tree_window_cap_fp8", op="attn_tree", B=4, T=24, Hkv=4, G=2, D=256, L=20011, spread=0.5, page=64,
             q="f32", cache="fp8", window=4096, cap=50.0, lens=13),
        # A tree of one chat: fp32 q, k, v as the products leave them.
        dict(name="append_tree_one", op="append_tree", B=1, T=16, Hq=32, Hkv=8, D=128, L=1000, page=16, x="f32", q="bf16",
             cache="bf16", norm=True, off=0.0, rot=128, inter=False, fused=False, lens=14),
        # Large trees of a batch into an 8-bit cache, one fused buffer, interleaved pairs on half of the head.
        dict(name="append_tree_batch", op="append_tree", B=48, T=63, Hq=32, Hkv=8, D=128, L=9001, page=32, x="bf16", q="bf16",
             cache="fp8", norm=True, off=1.0, rot=64, inter=True, fused=True, lens=15),
        # One chat's tree accepted: 36 layers' caches.
        dict(name="accept_one", op="accept", B=1, T=16, layers=36, Hkv=8, D=128, L=1000, page=16, cache="bf16", lens=16),
        # A batch's large trees: 30 layers' 8-bit caches.
        dict(name="accept_batch", op="accept", B=32, T=61, layers=30, Hkv=4, D=256, L=9001, page=32, cache="fp8", lens=17),
        # One token of a layer with 16 heads: fp32 rows as the products leave them.
        dict(name="latent_append_one", op="latent_append", B=1, T=1, H=16, latent=512, rope=64, L=1000, page=64, x="f32",
             cache="bf16", norm=True, inter=True, tree=False, lens=18),
        # Prompts on their way into an 8-bit cache.
        dict(name="latent_append_prompt", op="latent_append", B=4, T=2047, H=16, latent=512, rope=64, L=2047, page=64,
             x="bf16", cache="fp8", norm=True, inter=False, tree=False, lens=19),
        # One chat, a short history, 16 heads.
        dict(name="latent_attn_one", op="latent_attn", B=1, T=1, H=16, latent=512, rope=64, L=1000, spread=0.0, page=64,
             cache="bf16", tree=False, lens=20),
        # A serving batch of 128 heads whose histories differ a lot, empty slots among them.
        dict(name="latent_attn_batch", op="latent_attn", B=32, T=1, H=128, latent=512, rope=64, L=16001, spread=1.0, page=64,
             cache="bf16", tree=False, lens=21),
        # Trees of 9 drafted tokens over long documents in an 8-bit cache.
        dict(name="latent_attn_tree_long_fp8", op="latent_attn", B=2, T=9, H=16, latent=512, rope=64, L=65537, spread=0.3,
             page=32, cache="fp8", tree=True, lens=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_tree", "attn_tree", "append_tree", "accept", "latent_append", "latent_attn", "latent_attn"])
    lens, page = rng.randrange(1 << 20), rng.choice([8, 16, 32, 64, 128])
    cache = rng.choice(["bf16", "bf16", "fp8"])
    if op == "attn_tree":
        T = rng.choice([1, rng.randint(2, 16), rng.randint(2, 16), rng.randint(17, 64)])
        D = rng.choice([64, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        B = _log(rng, 1, 32)
        room = min(20_000_000, (8 * 61 * 32 * 128 * 6007 // 2) // (T * G))  # keys' values of all heads, and the scores' cost
        L = T + _log(rng, 1, max(2, min(60000, room // (B * Hkv * D))))
        return dict(op=op, B=B, T=T, Hkv=Hkv, G=G, D=D, L=L, spread=rng.choice([0.0, 0.5, 1.0]), page=page,
                    q=rng.choice(["bf16", "bf16", "f32"]), cache=cache, window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), lens=lens)
    if op == "append_tree":
        D, Hkv = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        T = rng.choice([1, rng.randint(2, 16), rng.randint(17, 64)])
        B = _log(rng, 1, max(1, min(256, 48 * 63 * 48 * 128 // (T * (Hq + 2 * Hkv) * D))))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, L=T + _log(rng, 1, 20000), page=page, x=rng.choice(["f32", "bf16"]),
                    q=rng.choice(["bf16", "bf16", "f32"]), cache=cache, norm=rng.random() < 0.6, off=rng.choice([0.0, 1.0]),
                    rot=rng.choice([D, D, D // 2]), inter=rng.random() < 0.4, fused=rng.random() < 0.5, lens=lens)
    if op == "accept":
        T, D = rng.choice([rng.randint(2, 16), rng.randint(17, 64)]), rng.choice([64, 128, 256])
        return dict(op=op, B=_log(rng, 1, 32), T=T, layers=rng.randint(1, 36), Hkv=rng.choice([1, 2, 4, 8]) * 64 // D or 1, D=D,
                    L=T + _log(rng, 1, 20000), page=page, cache=cache, lens=lens)
    latent, rope = rng.choice([(512, 64), (512, 64), (256, 64), (256, 32)])
    H = rng.choice([1, 4, 8, 16, 16, 20, 32, 40, 64, 128])
    if op == "latent_append":
        B = _log(rng, 1, 128)
        tree = rng.random() < 0.4
        most = max(1, 4 * 2000 * 17 * 576 // (B * (H + 1) * (latent + rope)))
        T = min(rng.randint(1, 64), most) if tree else min(4096, _log(rng, 1, most))
        return dict(op=op, B=B, T=T, H=H, latent=latent, rope=rope, L=T + _log(rng, 1, 20000), page=page,
                    x=rng.choice(["f32", "bf16"]), cache=cache, norm=rng.random() < 0.8, inter=rng.random() < 0.5, tree=tree,
                    lens=lens)
    tree = rng.random() < 0.4
    T = rng.choice([rng.randint(2, 16), rng.randint(17, 64)]) if tree else rng.choice([1, 1, 1, rng.randint(2, 16)])
    B = _log(rng, 1, 64)
    room = min(131071, (32 * 128 * 8000) // (T * H)) // B  # positions of all sequences, and the scores' cost
    L = T + _log(rng, 1, max(2, min(131071, room)))
    return dict(op=op, B=B, T=T, H=H, latent=latent, rope=rope, L=L, spread=rng.choice([0.0, 0.5, 1.0]), page=page,
                cache=cache, tree=tree, lens=lens)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


def _lengths(case):
    """The sequences' lengths, the new tokens included: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    T, L = case["T"], case["L"]
    if "spread" not in case:
        lens = [r.randint(T, L) for _ in range(case["B"])]
    else:
        lens = [max(T, int(L * (1.0 - case["spread"] * r.random()))) for _ in range(case["B"])]
        if case["spread"] == 1.0 and case["B"] >= 4:
            lens[r.randrange(case["B"])] = 0  # an empty slot of the batch
            lens[r.randrange(case["B"])] = T
    return lens


def _parents(case):
    """Each sequence's tree: every node's parent (-1: the root, node 0); None for padding.  Part of the case, as drafters
    take their trees' shapes from a table."""
    r = random.Random(case["lens"] + 7)
    out = []
    for n in _lengths(case):
        T = case["T"]
        nodes = 0 if n == 0 else T if r.random() < 0.5 else r.randint((T + 1) // 2, T)
        # nodes in the order of their depth, the likelier parents first
        depth, par = [0], [-1]
        wide = r.choice([2, 3, 5, 8])
        while len(par) < nodes:
            u = len(par)
            par.append(max(0, (u - 1) // wide - r.randrange(2)))
            depth.append(depth[par[-1]] + 1)
        out.append((par[:nodes] + [None] * (T - nodes))[:T])
    return out


def _masks(parents):
    rows = []
    for par in parents:
        m = []
        for t, p in enumerate(par):
            x = 0 if p is None else (1 << t) | (m[p] if p >= 0 else 0)
            m.append(x)
        rows.append([x - (1 << 64) if x >= 1 << 63 else x for x in m])
    return rows


def _branch(case):
    """The branch that each sequence's verification accepts: one whose nodes are in place already or lie behind the branch's
    new place, so that a pass can be repeated."""
    r = random.Random(case["lens"] + 9)
    out = []
    for par in _parents(case):
        paths = []
        for t, p in enumerate(par):
            if p is None:
                break
            paths.append((paths[p] if p >= 0 else []) + [t])
        good = [x for x in paths if all(u == i or u >= len(x) for i, u in enumerate(x))]
        longest = max((len(x) for x in good), default=0)
        out.append(r.choice([x for x in good if len(x) >= longest - 1]) if good else [])
    return out


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


def _paged(case, lens, g, whole):
    """A pool of pages in which the sequences' pages lie in any order, and the table of each sequence's pages; without
    `whole` only the pages that the new tokens lie in are present."""
    P, T = case["page"], case["T"]
    used = [-(-n // P) for n in lens]
    first = [0 if whole else max(0, n - T) // P for n in lens]
    need = [u - f for u, f in zip(used, first)]
    width, n_pages = max(1, max(used)), sum(need) + 3
    ids = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), width), 0, dtype=torch.int32, device="cuda")
    at = 0
    for b, (f, m) in enumerate(zip(first, need)):
        table[b, f:f + m] = ids[at:at + m]
        at += m
    return n_pages, table


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    s = dict(case)
    op, lens, ct = case["op"], _lengths(case), _TYPES[case["cache"]]
    B, T, P = case["B"], case["T"], case["page"]
    n_pages, s["table"] = _paged(case, lens, g, op in ("attn_tree", "latent_attn"))
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["masks"] = torch.tensor(_masks(_parents(case)), dtype=torch.int64, device="cuda") if case.get("tree", True) else None
    s["k_scale"], s["v_scale"] = (0.02, 0.015) if case["cache"] == "fp8" else (1.0, 1.0)
    up = (lambda scale: 1.0 / scale) if case["cache"] == "fp8" else (lambda scale: 1.0)
    if op in ("latent_append", "latent_attn"):
        return _prepare_latent(s, case, g, n_pages, ct, up)
    Hkv, D = case["Hkv"], case["D"]
    if op == "accept":
        shape = (case["layers"], n_pages, P, Hkv, D)
        s["k"], s["v"] = _randn(shape, ct, g, up(s["k_scale"])), _randn(shape, ct, g, up(s["v_scale"]))
        # drafted words, the children of a node all different; the model's word after each node: on the branch the next one's
        words = torch.argsort(torch.rand((B, 151936), device="cuda", generator=g), 1)[:, :2 * T].to(torch.int32)
        s["tokens"], s["ids"] = words[:, :T].contiguous(), words[:, T:].contiguous()
        for b, path in enumerate(_branch(case)):
            for u, w in zip(path, path[1:]):
                s["ids"][b, u] = s["tokens"][b, w]
        s["path"] = torch.empty((B, T), dtype=torch.int32, device="cuda")
        s["count"], s["next"], s["new_lens"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
        if own:
            from gguf_quant_weight_super_gb300 import kq
            s["set_h"] = kq.CacheSet([kq.KVCache(k, v, s["k_scale"], s["v_scale"]) for k, v in zip(s["k"], s["v"])])
        return s
    if op == "attn_tree":
        Hq = Hkv * case["G"]
        s["k"] = _randn((n_pages, P, Hkv, D), ct, g, up(s["k_scale"]))
        s["v"] = _randn((n_pages, P, Hkv, D), ct, g, up(s["v_scale"]))
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
        if op == "attn_tree":
            s["ws"] = kq.attn_tree_workspace(s["cache_h"], B, T, Hq)
        else:
            s["rope_h"] = kq.RopeNorm(s["table_cs"], interleaved=case["inter"], q_norm=s["wq"], k_norm=s["wk"],
                                      eps=s["eps"], norm_offset=case["off"])
    return s


def _prepare_latent(s, case, g, n_pages, ct, up):
    B, T, H, P, C, R = (case[n] for n in ("B", "T", "H", "page", "latent", "rope"))
    s["c_scale"] = s.pop("k_scale")
    s.pop("v_scale")
    if case["op"] == "latent_attn":
        s["c"] = _randn((n_pages, P, C + R), ct, g, up(s["c_scale"]))
        s["q"] = _randn((B, T, H, C + R), torch.bfloat16, g, 1.4)  # peaked scores
        s["scale"] = (128 + R) ** -0.5  # of the expanded heads
        s["out"] = torch.empty((B, T, H, C), dtype=torch.bfloat16, device="cuda")
    else:
        xt = _TYPES[case["x"]]
        s["c"] = torch.zeros((n_pages, P, C + R), dtype=ct, device="cuda")
        s["x"] = _randn((B, T, C + R), xt, g, 1.5)                 # latent | rope key, one product's row
        s["xq"] = _randn((B, T, H, C), xt, g, 1.5)                 # the queries, absorbed
        s["xr"] = _randn((B, T, H, 128 + R), xt, g, 1.5)[..., 128:]  # their rope parts, inside of the queries' product
        s["eps"] = 1e-6
        s["w"] = 1.0 + 0.2 * torch.randn(C, device="cuda", generator=g) if case["norm"] else None
        s["table_cs"] = _rope_table(case["L"], R)
        s["q"] = torch.empty((B, T, H, C + R), dtype=torch.bfloat16, device="cuda")
    if own:
        from gguf_quant_weight_super_gb300 import kq
        s["cache_h"] = kq.LatentCache(s["c"], C, s["c_scale"])
        if case["op"] == "latent_attn":
            s["ws"] = kq.latent_attn_workspace(s["cache_h"], B, T, H)
        else:
            s["rope_h"] = kq.RopeNorm(s["table_cs"], interleaved=case["inter"], k_norm=s["w"], eps=s["eps"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from gguf_quant_weight_super_gb300 import kq
    op = s["op"]
    if op == "attn_tree":
        return kq.attn_tree(s["cache_h"], s["table"], s["lens"], s["masks"], s["q"], s["ws"], scale=s["scale"],
                            softcap=s["cap"], window=s["window"], out=s["out"])
    if op == "append_tree":
        kq.kv_append_tree(s["cache_h"], s["table"], s["lens"], s["masks"], s["xq"], s["xk"], s["xv"], s["rope_h"],
                          q_out=s["q"])
        return {"q": s["q"], "k": s["k"], "v": s["v"]}
    if op == "accept":
        kq.tree_accept(s["set_h"], s["table"], s["lens"], s["masks"], s["tokens"], s["ids"], path=s["path"],
                       count=s["count"], next_ids=s["next"], new_lens=s["new_lens"])
        return {n: s[n] for n in ("path", "count", "next", "new_lens", "k", "v")}
    if op == "latent_append":
        kq.latent_append(s["cache_h"], s["table"], s["lens"], s["xq"], s["xr"], s["x"], s["rope_h"], tree=s["masks"],
                         q_out=s["q"])
        return {"q": s["q"], "c": s["c"]}
    return kq.latent_attn(s["cache_h"], s["table"], s["lens"], s["q"], s["ws"], s["scale"], tree=s["masks"], out=s["out"])


def _run_plain(s):
    return {"attn_tree": _plain_attn, "append_tree": _plain_append, "accept": _plain_accept,
            "latent_append": _plain_latent_append, "latent_attn": _plain_latent_attn}[s["op"]](s)


def _bits(masks):
    """[B, T, T]: whether token t sees drafted token u."""
    T = masks.shape[1]
    return ((masks[:, :, None] >> torch.arange(T, device="cuda")) & 1).bool()


def _tree(s):
    """Each new token's position (-1 for padding) and what it sees of the drafted tokens [B, T, T]."""
    T, base = s["T"], s["lens"][:, None].long() - s["T"]
    if s["masks"] is None:
        t = torch.arange(T, device="cuda")
        return torch.where(base + t >= 0, base + t, -1), (t <= t[:, None]).expand(len(base), T, T)
    bits = _bits(s["masks"]) & (base >= 0)[:, :, None]
    n = bits.sum(2)
    return torch.where(n > 0, base + n - 1, -1), bits


def _sees(s, L):
    """[B, T, L]: whether a token sees a position's slot."""
    at, bits = _tree(s)
    T = s["T"]
    j = torch.arange(L, device="cuda")
    base = (s["lens"].long() - T)[:, None]
    u = j - base                                                       # the drafted token in slot j
    drafted = bits.gather(2, u.clamp(0, T - 1)[:, None, :].expand(-1, T, -1)) & ((u >= 0) & (u < T))[:, None]
    see = ((u < 0)[:, None] & (at >= 0)[:, :, None]) | drafted
    if s.get("window"):
        where = torch.where(u < 0, j, at.gather(1, u.clamp(0, T - 1)))   # the slots' positions
        see = see & (where[:, None] > at[:, :, None] - s["window"])
    return see


def _weights(x, see):
    """softmax over what is seen; rows that see nothing: zeros."""
    x = x.masked_fill(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
    total = w.sum(-1, keepdim=True)
    return w / torch.where(total == 0, 1.0, total)


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
    w = _weights(x, _sees(s, L)[:, None, :, None, :])
    v = torch.where((torch.arange(L, device="cuda") < s["lens"][:, None])[:, :, None, None], v, 0.0)
    o = torch.matmul(w.view(B, Hkv, -1, L), v.permute(0, 2, 1, 3)).view(B, Hkv, T, -1, D)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(s["q"].dtype)


def _plain_latent_attn(s):
    B, T, H, W = s["q"].shape
    C, L = s["latent"], s["table"].shape[1] * s["page"]
    c = s["c"][s["table"]].float().view(B, L, W) * s["c_scale"]
    c = torch.where((torch.arange(L, device="cuda") < s["lens"][:, None])[:, :, None], c, 0.0)
    x = torch.matmul(s["q"].float().view(B, T * H, W), c.transpose(1, 2)).view(B, T, H, L) * s["scale"]
    w = _weights(x, _sees(s, L)[:, :, None, :])
    return torch.matmul(w.view(B, T * H, L), c[:, :, :C]).view(B, T, H, C).to(torch.bfloat16)


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


def _slots(s, at):
    """Where the new tokens go: pages and slots of those that are not padding, and which those are."""
    T, P = s["T"], s["page"]
    ok = at >= 0
    slot = (s["lens"][:, None].long() - T + torch.arange(T, device="cuda")).clamp(min=0)
    return s["table"].long().gather(1, slot // P)[ok], (slot % P)[ok], ok


def _plain_store(pool, x, where, scale):
    page, slot, ok = where
    x = x[ok] / scale
    pool[page, slot] = x.clamp(-448.0, 448.0).to(pool.dtype) if pool.dtype == torch.float8_e4m3fn else x.to(pool.dtype)


def _plain_append(s):
    rot = s["rot"]
    at, _ = _tree(s)
    where = _slots(s, at)
    cs = s["table_cs"][at.clamp(min=0)]
    c, sn = cs[:, :, None, :rot // 2], cs[:, :, None, rot // 2:]
    q = _plain_rotate(_plain_norm(s["xq"].float(), s["wq"], s["off"], s["eps"]), c, sn, rot, s["inter"])
    k = _plain_rotate(_plain_norm(s["xk"].float(), s["wk"], s["off"], s["eps"]), c, sn, rot, s["inter"])
    _plain_store(s["k"], k, where, s["k_scale"])
    _plain_store(s["v"], s["xv"].float(), where, s["v_scale"])
    q = torch.where((at >= 0)[:, :, None, None], q, 0.0)
    return {"q": q.to(s["q"].dtype), "k": s["k"], "v": s["v"]}


def _plain_latent_append(s):
    C, R = s["latent"], s["rope"]
    at, _ = _tree(s)
    where = _slots(s, at)
    cs = s["table_cs"][at.clamp(min=0)]
    c, sn = cs[:, :, None, :R // 2], cs[:, :, None, R // 2:]
    x = s["x"].float()
    key = _plain_rotate(x[:, :, None, C:], c, sn, R, s["inter"])[:, :, 0]
    _plain_store(s["c"], torch.cat([_plain_norm(x[..., :C], s["w"], 0.0, s["eps"]), key], -1), where, s["c_scale"])
    q = torch.cat([s["xq"].float(), _plain_rotate(s["xr"].float(), c, sn, R, s["inter"])], -1)
    q = torch.where((at >= 0)[:, :, None, None], q, 0.0)
    return {"q": q.to(torch.bfloat16), "c": s["c"]}


def _plain_accept(s):
    B, T, P = s["B"], s["T"], s["page"]
    bits = _bits(s["masks"])
    there = bits[:, 0, 0] & (s["lens"] >= T)                                   # whether there is a root at all
    one = torch.eye(T, dtype=torch.bool, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = torch.where(there, 0, -1)
    count, nxt = there.int(), s["ids"][:, 0].clone()
    going, rows = there, torch.arange(B, device="cuda")
    for i in range(1, T):
        child = (bits == (bits[rows, cur][:, None] | one)).all(2)             # the current node's children
        child &= (torch.arange(T, device="cuda") != cur[:, None]) & (s["tokens"] == nxt[:, None]) & going[:, None]
        going = child.any(1)
        cur = torch.where(going, child.int().argmax(1), cur)
        path[:, i] = torch.where(going, cur, -1)
        count = count + going
        nxt = s["ids"][rows, cur]
    base = (s["lens"].long() - T).clamp(min=0)
    i = torch.arange(T, device="cuda")
    move = (path >= 0) & (path != i)
    to, frm = (base[:, None] + i)[move], (base[:, None] + path.long())[move]
    table = s["table"].long()
    row = rows[:, None].expand(B, T)[move]
    tp, fp = table[row, to // P], table[row, frm // P]
    for pool in (s["k"], s["v"]):
        raw = pool.view(torch.int16 if pool.dtype == torch.bfloat16 else torch.uint8)
        raw[:, tp, to % P] = raw[:, fp, frm % P]
    return {"path": path, "count": count.int(), "next": torch.where(there, nxt, -1), "new_lens": (base + count).int(),
            "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def _pairs(case):
    """(slots that some new token sees, (token, slot) pairs) of all sequences."""
    union, pairs, T, W = 0, 0, case["T"], case.get("window", 0)
    masks = _masks(_parents(case)) if case.get("tree", True) else None
    for b, n in enumerate(_lengths(case)):
        base = n - T
        if masks is None:
            union += n
            pairs += sum(max(0, base + t + 1) for t in range(T))
            continue
        if n == 0:
            continue
        least, drafted = base, 0
        for m in masks[b]:
            bits = bin(m & ((1 << 64) - 1)).count("1")
            if bits:
                seen = min(base, max(0, W - bits)) if W else base  # of the context
                least = min(least, base - seen)
                pairs += seen + (min(bits, W) if W else bits)
                drafted += 1
        union += base - least + drafted
    return union, pairs


def work(case):
    op, lens, T, size = case["op"], _lengths(case), case["T"], _BYTES[case["cache"]]
    ints = sum(-(-n // case["page"]) for n in lens) * 4 + 8 * case["B"] * T
    n = case["B"] * T
    if op == "append_tree":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        return {"bytes": n * (Hq + 2 * Hkv) * D * _BYTES[case["x"]] + n * case["rot"] * 4 + n * Hq * D * _BYTES[case["q"]]
                + 2 * n * Hkv * D * size, "flops": 10.0 * n * (Hq + Hkv) * D}
    if op == "latent_append":
        H, C, R = case["H"], case["latent"], case["rope"]
        return {"bytes": n * (H + 1) * (C + R) * _BYTES[case["x"]] + n * R * 4 + n * H * (C + R) * 2 + n * (C + R) * size,
                "flops": n * (6.0 * C + 6.0 * (H + 1) * R)}
    if op == "accept":
        moved = sum(sum(u != i for i, u in enumerate(p)) for p in _branch(case))
        return {"bytes": 2 * 2 * moved * case["layers"] * case["Hkv"] * case["D"] * size + 20 * n + 16 * case["B"],
                "flops": 4.0 * n}
    union, pairs = _pairs(case)
    if op == "attn_tree":
        Hkv, G, D = case["Hkv"], case["G"], case["D"]
        return {"bytes": 2 * union * Hkv * D * size + 2 * n * Hkv * G * D * _BYTES[case["q"]] + ints,
                "flops": 4.0 * pairs * Hkv * G * D}
    H, C, R = case["H"], case["latent"], case["rope"]
    return {"bytes": union * (C + R) * size + n * H * (2 * C + R) * 2 + ints, "flops": 2.0 * pairs * H * (2 * C + R)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn_tree": _exact_attn, "append_tree": _exact_append, "accept": _exact_accept,
            "latent_append": _exact_latent_append, "latent_attn": _exact_latent_attn}[case["op"]](case, s)


def _nodes(case):
    """Per sequence: its length, and for each new token that is not padding (token, position, drafted tokens it sees)."""
    T, out = case["T"], []
    parents = _parents(case) if case.get("tree", True) else None
    for b, n in enumerate(_lengths(case)):
        base, rows, seen = n - T, [], {}
        for t in range(T if n else 0):
            p = t - 1 if parents is None else parents[b][t]
            if p is None:
                continue
            seen[t] = (seen[p] if p >= 0 else []) + [t]
            rows.append((t, base + len(seen[t]) - 1, seen[t]))
        out.append((n, rows))
    return out


def _exact_attn(case, s):
    B, T, Hq, D = s["q"].shape
    Hkv, P, G, W = case["Hkv"], case["page"], case["G"], case["window"]
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    for b, (n, rows) in enumerate(_nodes(case)):
        if not rows:
            continue
        where = {t: p for t, p, _ in rows}
        lo = max(0, n - T - W + 1) if W else 0
        j = torch.arange(lo, n, device="cuda")
        pages = s["table"][b].long()[j // P]
        cols = [torch.tensor([x for x in range(max(lo, p - W + 1) if W else 0, n - T)]
                             + [n - T + u for u in seen if not W or where[u] > p - W], device="cuda") - lo for t, p, seen in rows]
        for h in range(Hkv):
            k = s["k"][:, :, h][pages, j % P].double() * s["k_scale"]
            v = s["v"][:, :, h][pages, j % P].double() * s["v_scale"]
            q = s["q"][b, :, h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,jd->tgj", q, k) * s["scale"]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            for (t, _, _), c in zip(rows, cols):
                out[b, t, h * G:(h + 1) * G] = torch.softmax(x[t][:, c], -1) @ v[c]
    return out


def _exact_latent_attn(case, s):
    B, T, H, _ = s["q"].shape
    C, P = case["latent"], case["page"]
    out = torch.zeros((B, T, H, C), dtype=torch.float64, device="cuda")
    for b, (n, rows) in enumerate(_nodes(case)):
        if not rows:
            continue
        j = torch.arange(n, device="cuda")
        c = s["c"][s["table"][b].long()[j // P], j % P].double() * s["c_scale"]
        for t, _, seen in rows:
            x = s["q"][b, t].double() @ c.T * s["scale"]
            hide = torch.ones(n, dtype=torch.bool, device="cuda")
            hide[:n - T] = False
            hide[torch.tensor([n - T + u for u in seen], device="cuda")] = False
            out[b, t] = torch.softmax(x.masked_fill(hide, float("-inf")), -1) @ c[:, :C]
    return out


def _turn(x, cs, first, second):
    half = cs.shape[1] // 2
    cos, sin = cs[:, :half].double()[:, None], cs[:, half:].double()[:, None]
    y = x.clone()
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y


def _pairs_of(rot, inter):
    first = torch.arange(rot // 2, device="cuda") * (2 if inter else 1)
    return first, first + (1 if inter else rot // 2)


def _exact_append(case, s):
    T, P, D = case["T"], case["page"], case["D"]
    k_pool, v_pool = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    qs = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (n, rows) in enumerate(_nodes(case)):
        t = torch.tensor([r[0] for r in rows], device="cuda")
        cs = s["table_cs"][torch.tensor([r[1] for r in rows], device="cuda")]
        turned = []
        for x, w in ((s["xq"][b], s["wq"]), (s["xk"][b], s["wk"])):
            x = x[t].double()
            if w is not None:
                x = x / (x.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * (w.double() + case["off"])
            turned.append(_turn(x, cs, *_pairs_of(case["rot"], case["inter"])))
        qs[b, t] = turned[0]
        slot = n - T + t
        where = (s["table"][b].long()[slot // P], slot % P)
        k_pool[where] = turned[1] / s["k_scale"]
        v_pool[where] = s["xv"][b][t].double() / s["v_scale"]
    if case["cache"] == "fp8":
        k_pool.clamp_(-448, 448), v_pool.clamp_(-448, 448)
    return {"q": qs, "k": k_pool, "v": v_pool}


def _exact_latent_append(case, s):
    T, P, C, R = case["T"], case["page"], case["latent"], case["rope"]
    pool = torch.zeros(s["c"].shape, dtype=torch.float64, device="cuda")
    qs = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    pairs = _pairs_of(R, case["inter"])
    for b, (n, rows) in enumerate(_nodes(case)):
        t = torch.tensor([r[0] for r in rows], device="cuda")
        cs = s["table_cs"][torch.tensor([r[1] for r in rows], device="cuda")]
        x = s["x"][b, t].double()
        latent = x[:, :C]
        if s["w"] is not None:
            latent = latent / (latent.square().sum(-1, keepdim=True) / C + s["eps"]).sqrt() * s["w"].double()
        slot = n - T + t
        pool[s["table"][b].long()[slot // P], slot % P] = torch.cat(
            [latent, _turn(x[:, None, C:], cs, *pairs)[:, 0]], 1) / s["c_scale"]
        qs[b, t] = torch.cat([s["xq"][b, t].double(), _turn(s["xr"][b, t].double(), cs, *pairs)], -1)
    if case["cache"] == "fp8":
        pool.clamp_(-448, 448)
    return {"q": qs, "c": pool}


def _exact_accept(case, s):
    """The branch that the model's words were made to follow, and the copies it takes, one slot after the other."""
    B, T, P = case["B"], case["T"], case["page"]
    path = torch.full((B, T), -1, dtype=torch.int32)
    count, nxt, new = ([0] * B for _ in range(3))
    k, v, table = s["k"].clone(), s["v"].clone(), s["table"].tolist()
    for b, (n, p) in enumerate(zip(_lengths(case), _branch(case))):
        base = max(0, n - T)
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        count[b], nxt[b], new[b] = len(p), int(s["ids"][b, p[-1]]) if p else -1, base + len(p)
        for i, u in enumerate(p):
            if u != i:
                to, frm = base + i, base + u
                for pool in (k, v):
                    pool[:, table[b][to // P], to % P] = pool[:, table[b][frm // P], frm % P]
    ints = [torch.tensor(x, dtype=torch.int32) for x in (count, nxt, new)]
    return {"path": path, "count": ints[0], "next": ints[1], "new_lens": ints[2], "k": k.double(), "v": v.double()}
