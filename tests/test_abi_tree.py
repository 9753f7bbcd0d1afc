"""CPU checks of what the calls for trees of drafted tokens and for latent caches refuse, before any CUDA call, and of the
binding's own checks of shapes and types."""
import ctypes

import pytest
import torch

from gguf_quant_weight_super_gb300 import kq
from tests.test_abi_decode import (ALIGN, ARG, CACHE_REFUSALS, F, L, SHAPE, UNSUPPORTED, WORKSPACE, cache,  # noqa: F401
                                   rope)


def latent(**kw):
    a = dict(dtype=1, latent_dim=512, rope_dim=64, page_size=16, n_pages=10, page_stride=16 * 576, slot_stride=576, c=F,
             scale=1.0)
    a.update(kw)
    return kq.KqLatentCache(*a.values())


LATENT_REFUSALS = [(dict(dtype=0), ARG), (dict(dtype=3), ARG), (dict(n_pages=-1), ARG), (dict(page_size=0), ARG),
                   (dict(page_size=24), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
                   (dict(latent_dim=384), UNSUPPORTED), (dict(rope_dim=0), UNSUPPORTED), (dict(rope_dim=96), UNSUPPORTED),
                   (dict(c=None), ARG), (dict(c=F + 8), ALIGN), (dict(slot_stride=580), ALIGN),
                   (dict(page_stride=-8), ALIGN), (dict(dtype=2, slot_stride=584), ALIGN), (dict(scale=0.0), ARG),
                   (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG)]
TREE_REFUSALS = [(dict(tree=None), ARG), (dict(tree=F + 4), ALIGN), (dict(T=65), UNSUPPORTED), (dict(T=-1), ARG),
                 (dict(B=-1), ARG), (dict(B=0), 0), (dict(T=0), 0), (dict(W=-1), ARG), (dict(lens=None), ARG),
                 (dict(table=None), ARG), (dict(lens=F + 2), ALIGN), (dict(table=F + 1), ALIGN)]


def test_append_tree_refusals(L):  # noqa: F811
    def call(c=None, r=None, **kw):
        a = dict(table=F, W=4, lens=F, tree=F, B=2, T=3, q=F, k=F, v=F, xd=1, qs=1024, ks=256, vs=256, Hq=8)
        a.update(kw)
        c, r = c or cache(), r or rope()
        return L.kq_kv_append_tree(ctypes.addressof(c), *a.values(), ctypes.addressof(r), F, 1, None)
    assert L.kq_kv_append_tree(None, F, 4, F, F, 2, 3, F, F, F, 1, 1024, 256, 256, 8, None, F, 1, None) == ARG
    for kw, want in CACHE_REFUSALS:
        assert call(cache(**kw)) == want, kw
    for kw, want in TREE_REFUSALS + [(dict(q=F + 4), ALIGN), (dict(xd=2), ARG), (dict(Hq=0), ARG), (dict(ks=-256), ALIGN)]:
        assert call(**kw) == want, kw
    assert call(r=rope(rot_dim=12)) == SHAPE and call(r=rope(cos_sin=None)) == ARG


def test_attn_tree_refusals(L):  # noqa: F811
    def call(c=None, **kw):
        a = dict(table=F, W=4, lens=F, tree=F, B=2, T=3, q=F, qd=1, qs=1024, Hq=8, scale=0.1, cap=0.0, window=0, out=F, ws=F,
                 wsb=1 << 40)
        a.update(kw)
        c = c or cache()
        return L.kq_attn_tree(ctypes.addressof(c), *a.values(), None)
    for kw, want in CACHE_REFUSALS:
        assert call(cache(**kw)) == want, kw
    for kw, want in TREE_REFUSALS + [(dict(qd=2), ARG), (dict(B=5000), UNSUPPORTED), (dict(Hq=7), ARG),
                                     (dict(Hq=34), UNSUPPORTED), (dict(cap=-1.0), ARG), (dict(scale=float("nan")), ARG),
                                     (dict(scale=float("inf")), ARG), (dict(window=-1), ARG), (dict(q=None), ARG),
                                     (dict(out=F + 4), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=F + 16), WORKSPACE),
                                     (dict(wsb=16), WORKSPACE), (dict(W=1 << 40), UNSUPPORTED)]:
        assert call(**kw) == want, kw
    size, c = L.kq_attn_tree_workspace_size, cache()
    c_ref = ctypes.addressof(c)
    assert size(c_ref, 2, 64, 8) > 0 and size(c_ref, 2, 65, 8) == 0 and size(c_ref, 2, 3, 7) == 0 and size(None, 2, 3, 8) == 0
    for hq in (2, 8, 32):  # room for any smaller T, and for chains
        for t in range(17):
            assert size(c_ref, 2, 16, hq) >= size(c_ref, 2, t, hq) >= L.kq_attn_workspace_size(c_ref, 2, t, hq)
    assert L.kq_attn_decode(c_ref, F, 4, F, 2, 17, F, 1, 1024, 8, 0.1, 0.0, 0, F, F, 1 << 40, None) == UNSUPPORTED


def test_accept_refusals(L):  # noqa: F811
    def call(fn, caches, n=None, **kw):
        a = dict(table=F, W=4, lens=F, tree=F, tokens=F, ids=F, B=2, T=3, path=F, count=F, next=F, new=F + 64)
        a.update(kw)
        kind = type(caches[0]) if caches else kq.KqKvCache
        arr = (kind * max(1, len(caches)))(*caches)
        return fn(ctypes.addressof(arr) if caches else None, len(caches) if n is None else n, *a.values(), None)
    for fn, one, refusals, most in ((L.kq_tree_accept, cache, CACHE_REFUSALS, 128),
                                    (L.kq_latent_accept, latent, LATENT_REFUSALS, 256)):
        for kw, want in refusals:
            assert call(fn, [one(), one(**kw)]) in (want, ARG) and call(fn, [one(**kw)]) == want, kw
        for kw, want in TREE_REFUSALS + [(dict(tokens=None), ARG), (dict(ids=None), ARG), (dict(tokens=F + 1), ALIGN),
                                         (dict(path=F + 2), ALIGN), (dict(new=F), ARG), (dict(B=65536), UNSUPPORTED)]:
            assert call(fn, [one(), one()], **kw) == want, kw
        assert call(fn, [], n=1) == ARG and call(fn, [one()], n=-1) == ARG
        assert call(fn, [one()] * (most + 1)) == UNSUPPORTED
        assert call(fn, [one(), one(n_pages=9)]) == ARG and call(fn, [one(), one(page_size=8)]) == ARG
        assert call(fn, [], B=0) == 0 and call(fn, [], tokens=None) == ARG
    assert call(L.kq_tree_accept, [cache(), cache(dtype=2)]) == ARG
    assert call(L.kq_latent_accept, [latent(), latent(slot_stride=592)]) == ARG


def test_accept_refuses_overlaps(L):  # noqa: F811
    """Blocks walk and move by themselves: outputs over inputs, and one pool twice, would depend on their order."""
    ins = dict(table=F + 1024, W=4, lens=F + 2048, tree=F + 3328, tokens=F + 4096, ids=F + 5120, B=2, T=3)
    outs = dict(path=F + 6144, count=F + 7168, next=F + 8192, new=F + 9216)
    two = (kq.KqKvCache * 2)(cache(k=F, v=F + (1 << 20)), cache(k=F + (2 << 20), v=F + (1 << 20)))
    assert L.kq_tree_accept(ctypes.addressof(two), 2, *ins.values(), *outs.values(), None) == ARG
    two = (kq.KqLatentCache * 2)(latent(), latent())
    assert L.kq_latent_accept(ctypes.addressof(two), 2, *ins.values(), *outs.values(), None) == ARG
    for o in outs:
        for i in ("table", "lens", "tree", "tokens", "ids"):
            assert L.kq_tree_accept(None, 0, *ins.values(), *{**outs, o: ins[i]}.values(), None) == ARG, (o, i)


def test_latent_refusals(L):  # noqa: F811
    def append(c=None, r=None, **kw):
        a = dict(table=F, W=4, lens=F, tree=F, B=2, T=3, ql=F, qr=F, rows=F, xd=1, ls=512, rs=64, hs=64, cs=576, H=8)
        a.update(kw)
        c, r = c or latent(), r or rope(q_norm=None, rot_dim=64)
        return L.kq_latent_append(ctypes.addressof(c), *a.values(), ctypes.addressof(r), kw.get("out", F), None)

    def attn(c=None, **kw):
        a = dict(table=F, W=4, lens=F, tree=F, B=2, T=3, q=F, qs=4608, H=8, scale=0.1, out=F, ws=F, wsb=1 << 40)
        a.update(kw)
        c = c or latent()
        return L.kq_latent_attn(ctypes.addressof(c), *a.values(), None)
    for call in (append, attn):
        for kw, want in LATENT_REFUSALS:
            assert call(latent(**kw)) == want, kw
        for kw, want in TREE_REFUSALS[1:]:
            assert call(**kw) == want, kw
    for kw, want in [(dict(xd=2), ARG), (dict(H=0), ARG), (dict(ql=None), ARG), (dict(qr=None), ARG), (dict(rows=None), ARG),
                     (dict(ql=F + 8), ALIGN), (dict(qr=F + 4), ALIGN), (dict(rs=65), ALIGN), (dict(hs=-64), ALIGN),
                     (dict(tree=None, B=1 << 20, T=1 << 10), UNSUPPORTED), (dict(tree=None, T=65, ql=None), ARG)]:
        assert append(**kw) == want, kw
    base = dict(q_norm=None, rot_dim=64)
    for kw, want in [(dict(q_norm=F), ARG), (dict(rot_dim=32), SHAPE), (dict(rot_dim=0), SHAPE), (dict(cos_sin=None), ARG),
                     (dict(k_norm=F + 4), ALIGN), (dict(cos_sin=F + 8), ALIGN), (dict(n_positions=-1), ARG)]:
        assert append(r=rope(**{**base, **kw})) == want, kw
    for kw, want in [(dict(H=0), ARG), (dict(H=257), UNSUPPORTED), (dict(B=5000), UNSUPPORTED), (dict(tree=None, T=65), UNSUPPORTED),
                     (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(q=None), ARG), (dict(out=None), ARG),
                     (dict(q=F + 8), ALIGN), (dict(qs=4604), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=F + 128), WORKSPACE),
                     (dict(wsb=8), WORKSPACE), (dict(W=1 << 40), UNSUPPORTED), (dict(W=1 << 28, H=256, T=64), UNSUPPORTED)]:
        assert attn(**kw) == want, kw
    size, c = L.kq_latent_attn_workspace_size, latent()
    assert size(ctypes.addressof(c), 2, 64, 128) > 0 and size(ctypes.addressof(c), 2, 65, 128) == 0
    assert size(ctypes.addressof(latent(latent_dim=100)), 2, 3, 8) == 0 and size(None, 2, 3, 8) == 0


def test_binding_refusals(L):  # noqa: F811
    c = torch.zeros((4, 8, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kq.LatentCache(c, 512)                          # host tensor
    with pytest.raises(ValueError):
        kq.LatentCache(c, 576)
    with pytest.raises(ValueError):
        kq.LatentCache(c.transpose(1, 2), 512)
    with pytest.raises(TypeError):
        kq.LatentCache(c.float(), 512)
    with pytest.raises(TypeError):
        kq.CacheSet([object()])
    i32, i64 = torch.int32, torch.int64
    table, lens = torch.zeros((2, 3), dtype=i32), torch.zeros(2, dtype=i32)
    for tree in (torch.zeros((2, 4), dtype=i32), torch.zeros((2, 5), dtype=i64), torch.zeros((4, 2), dtype=i64).T):
        with pytest.raises(ValueError):
            kq._tables(table, lens, tree, 2, 4)
    with pytest.raises(ValueError):
        kq._tables(table.long(), lens, None, 2, 4)
    assert kq._tables(table, lens, torch.zeros((2, 4), dtype=i64), 2, 4) == (False, 3)
    tree, words = torch.zeros((2, 4), dtype=i64), torch.zeros((2, 4), dtype=i32)
    with pytest.raises(ValueError):
        kq.tree_accept(kq.CacheSet([]), table, lens, tree, words.long(), words)
    with pytest.raises(ValueError):
        kq.tree_accept(kq.CacheSet([]), table, lens, tree, words, words)  # host tensors


def test_an_empty_batch_takes_every_length_that_a_tree_can_have(L):  # noqa: F811
    """An empty tensor's address is NULL."""
    c, r = cache(), rope()
    c_ref, r_ref = ctypes.addressof(c), ctypes.addressof(r)
    for tree in (None, F):
        for T in (0, 1, 16, 17, 61, 64):
            assert L.kq_attn_tree(c_ref, F, 4, F, tree, 0, T, F, 1, 1024, 8, 0.1, 0.0, 0, F, F, 1 << 40, None) == 0, (tree, T)
            assert L.kq_kv_append_tree(c_ref, F, 4, F, tree, 0, T, F, F, F, 1, 1024, 256, 256, 8, r_ref, F, 1, None) == 0
            assert L.kq_tree_accept(c_ref, 1, F, 4, F, tree, F, F, 0, T, F, F, F, F + 64, None) == 0
        assert L.kq_attn_tree(c_ref, F, 4, F, tree, 0, 65, F, 1, 1024, 8, 0.1, 0.0, 0, F, F, 1 << 40, None) == UNSUPPORTED
    assert L.kq_attn_decode(c_ref, F, 4, F, 0, 17, F, 1, 1024, 8, 0.1, 0.0, 0, F, F, 1 << 40, None) == UNSUPPORTED
