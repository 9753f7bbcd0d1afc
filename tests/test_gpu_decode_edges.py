"""kq_kv_append, kq_attn_decode and kq_sample where calls meet: one workspace for many calls, tensors on other streams, and
arguments at the ends of their types.  The 64-bit definitions and the bounds are test_gpu_cache.py's."""
import pytest
import torch

from gguf_quant_weight_super_gb300 import kq
from tests.gpu_util import require_gpu
from tests.test_gpu_cache import BF16, F8, F32, Paged, rand_q

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
