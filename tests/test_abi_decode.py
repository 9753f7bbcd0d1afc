"""CPU checks of what kq_kv_append, kq_attn_decode and kq_sample refuse, before any CUDA call, and of the binding's own
checks of shapes and types."""
import ctypes

import pytest
import torch

from gguf_quant_weight_super_gb300 import build as kqbuild
from gguf_quant_weight_super_gb300 import kq

F = 0x100000
ARG, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = -1, -3, -4, -5, -7


@pytest.fixture(scope="module")
def L():
    kqbuild.build()
    return kq.lib()


def cache(**kw):
    a = dict(dtype=1, n_kv_heads=2, head_dim=128, page_size=16, n_pages=10, page_stride=4096, slot_stride=256,
             head_stride=128, k=F, v=F, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return kq.KqKvCache(*a.values())


def rope(**kw):
    a = dict(q_norm=F, k_norm=F, eps=1e-6, norm_offset=0.0, cos_sin=F, n_positions=100, rot_dim=128, interleaved=0)
    a.update(kw)
    return kq.KqRope(*a.values())


CACHE_REFUSALS = [(dict(dtype=0), ARG), (dict(dtype=3), ARG), (dict(n_kv_heads=0), ARG), (dict(n_pages=-1), ARG),
                  (dict(page_size=0), ARG), (dict(page_size=24), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
                  (dict(head_dim=80), UNSUPPORTED), (dict(k=None), ARG), (dict(v=None), ARG), (dict(k=F + 8), ALIGN),
                  (dict(v=F + 2), ALIGN), (dict(slot_stride=260), ALIGN), (dict(head_stride=-128), ALIGN),
                  (dict(page_stride=4097), ALIGN), (dict(dtype=2, slot_stride=264), ALIGN), (dict(k_scale=0.0), ARG),
                  (dict(v_scale=-1.0), ARG), (dict(k_scale=float("nan")), ARG), (dict(v_scale=float("inf")), ARG)]


def append(L, c=None, r=None, null_cache=False, null_rope=False, **kw):
    c, r = c or cache(), r or rope()
    a = dict(table=F, W=4, lens=F, B=2, T=3, q=F, k=F, v=F, xd=1, qs=1024, ks=256, vs=256, Hq=8)
    a.update({k: v for k, v in kw.items() if k in a})
    out, od = kw.get("out", F), kw.get("od", 1)
    return L.kq_kv_append(None if null_cache else ctypes.addressof(c), *a.values(),
                          None if null_rope else ctypes.addressof(r), out, od, None)


def test_append_refusals(L):
    assert append(L, null_cache=True) == ARG and append(L, null_rope=True) == ARG
    for kw, want in CACHE_REFUSALS:
        assert append(L, cache(**kw)) == want, kw
    for kw, want in [(dict(xd=2), ARG), (dict(od=2), ARG), (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(Hq=0), ARG),
                     (dict(W=-1), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(q=None), ARG),
                     (dict(out=None), ARG), (dict(q=F + 4), ALIGN), (dict(out=F + 8), ALIGN), (dict(qs=1001), ALIGN),
                     (dict(ks=-256), ALIGN), (dict(table=F + 2), ALIGN), (dict(B=0), 0), (dict(T=0), 0),
                     (dict(B=1 << 20, T=1 << 10), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED)]:
        assert append(L, **kw) == want, kw
    for kw, want in [(dict(rot_dim=12), SHAPE), (dict(rot_dim=136), SHAPE), (dict(rot_dim=-8), ARG),
                     (dict(n_positions=-1), ARG), (dict(cos_sin=None), ARG), (dict(cos_sin=F + 4), ALIGN),
                     (dict(q_norm=F + 4), ALIGN), (dict(k_norm=F + 8), ALIGN)]:
        assert append(L, r=rope(**kw)) == want, kw


def attn(L, c=None, null_cache=False, **kw):
    c = c or cache()
    a = dict(table=F, W=4, lens=F, B=2, T=3, q=F, qd=1, qs=1024, Hq=8, scale=0.1, cap=0.0, window=0, out=F, ws=F,
             wsb=1 << 40)
    a.update(kw)
    return L.kq_attn_decode(None if null_cache else ctypes.addressof(c), *a.values(), None)


def test_attn_refusals(L):
    assert attn(L, null_cache=True) == ARG
    for kw, want in CACHE_REFUSALS:
        assert attn(L, cache(**kw)) == want, kw
    for kw, want in [(dict(qd=2), ARG), (dict(B=-1), ARG), (dict(T=17), UNSUPPORTED), (dict(B=5000), UNSUPPORTED),
                     (dict(Hq=7), ARG), (dict(Hq=0), ARG), (dict(Hq=34), UNSUPPORTED), (dict(W=-1), ARG),
                     (dict(cap=-1.0), ARG), (dict(cap=float("nan")), ARG), (dict(scale=float("nan")), ARG),
                     (dict(window=-1), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(q=None), ARG),
                     (dict(out=None), ARG), (dict(q=F + 8), ALIGN), (dict(out=F + 4), ALIGN), (dict(qs=1004), ALIGN),
                     (dict(lens=F + 1), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=F + 16), WORKSPACE),
                     (dict(wsb=16), WORKSPACE), (dict(B=0), 0), (dict(T=0), 0)]:
        assert attn(L, **kw) == want, kw
    c = cache()
    size = L.kq_attn_workspace_size
    assert size(ctypes.addressof(c), 2, 3, 8) > 0 and size(ctypes.addressof(c), 2, 17, 8) == 0
    assert size(ctypes.addressof(c), 2, 3, 7) == 0 and size(None, 2, 3, 8) == 0
    assert size(ctypes.addressof(cache(head_dim=96)), 2, 3, 8) == 0


def test_sample_refusals(L):
    def call(**kw):
        a = dict(x=F, dt=0, stride=1000, M=2, V=1000, u=F, t=F, k=F, p=F, mp=F, ids=F, probs=F, ws=F, wsb=1 << 40)
        a.update(kw)
        return L.kq_sample(*a.values(), None)
    for kw, want in [(dict(dt=2), ARG), (dict(M=-1), ARG), (dict(V=-1), ARG), (dict(stride=-1), ARG), (dict(x=None), ARG),
                     (dict(u=None), ARG), (dict(ids=None), ARG), (dict(V=0), UNSUPPORTED),
                     (dict(V=(1 << 20) + 1), UNSUPPORTED), (dict(M=0), 0), (dict(x=F + 2), ALIGN),
                     (dict(dt=1, x=F + 1), ALIGN), (dict(t=F + 2), ALIGN), (dict(k=F + 1), ALIGN), (dict(ids=F + 2), ALIGN),
                     (dict(probs=F + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=F + 128), WORKSPACE),
                     (dict(wsb=8), WORKSPACE)]:
        assert call(**kw) == want, kw
    assert L.kq_sample_workspace_size(2, 1000) > 0
    assert L.kq_sample_workspace_size(-1, 1000) == 0 and L.kq_sample_workspace_size(1, 0) == 0


def test_binding_refusals(L):
    x = torch.zeros((4, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kq.KVCache(x, x)                                   # host tensors
    with pytest.raises(ValueError):
        kq.KVCache(x, x[:2])
    with pytest.raises(ValueError):
        kq.KVCache(x.transpose(2, 3), x.transpose(2, 3))   # last dimension not contiguous
    with pytest.raises(TypeError):
        kq.KVCache(x.float(), x.float())
    with pytest.raises(TypeError):
        kq.RopeNorm(torch.zeros((4, 8), dtype=torch.float64))
    with pytest.raises(ValueError):
        kq._rows("q", torch.zeros(2, 3, 4, 64), 2, 3, 128)
    with pytest.raises(ValueError):
        kq._rows("q", torch.zeros(2, 4, 3, 64).transpose(1, 2), 2, 3, 64)
    assert kq._rows("q", torch.zeros(2, 3, 6, 64)[:, :, :4], 2, 3, 64) == (4, 384)
    with pytest.raises(ValueError):
        kq.sample(torch.zeros(3, 5), torch.zeros(2))
    with pytest.raises(ValueError):
        kq.sample(torch.zeros(5, 3).T, torch.zeros(3))


def test_attn_refuses_scales_and_caps_that_are_not_finite(L):
    """An infinite cap or scale would make every score that is 0 a NaN."""
    inf = float("inf")
    for kw in (dict(cap=inf), dict(scale=inf), dict(scale=-inf)):
        assert attn(L, **kw) == ARG, kw
    for kw in (dict(cap=30.0), dict(scale=0.0), dict(scale=-0.5), dict(cap=3e38)):
        assert attn(L, ws=None, **kw) == WORKSPACE, kw  # past these checks
