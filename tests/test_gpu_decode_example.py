"""examples/decode_step.py: the last logits of a generation (prompt blocks, then single tokens, through the paged caches)
against a dense recomputation of the whole text from dequantized weights in 64 bits."""
import importlib.util
import os

import pytest
import torch

from gguf_quant_weight_super_gb300 import kq, synth
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    from gguf_quant_weight_super_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense_logits(d, tokens):
    """[B, V] after the whole text, no cache."""
    B, L = tokens.shape

    def weight(w):
        n, k = w[1], w[2]
        return kq.dequant(synth.Q4_K, w[0], n * k).view(n, k).double()

    def norm(x):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)

    def turn(x, table, w):
        x = norm(x) * w.double()
        c, s = table[:L, None, :64].double(), table[:L, None, 64:].double()
        a, b = x[..., :64], x[..., 64:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    x = d.embedding[tokens].double()
    mask = torch.full((L, L), float("-inf"), dtype=torch.float64, device="cuda").triu(1)
    for w in d.layers:
        h = norm(x)
        q, k, v = ((h @ weight(w[n]).T).view(B, L, -1, d.D) for n in ("q", "k", "v"))
        q, k = turn(q, w["rope"].cos_sin, w["rope"].q_norm), turn(k, w["rope"].cos_sin, w["rope"].k_norm)
        k, v = (t.repeat_interleave(d.heads // d.kv, 2) for t in (k, v))
        p = torch.softmax(torch.einsum("bihd,bjhd->bhij", q, k) * d.D ** -0.5 + mask, -1)
        x = x + torch.einsum("bhij,bjhd->bihd", p, v).reshape(B, L, -1) @ weight(w["o"]).T
        h = norm(x)
        x = x + (torch.nn.functional.silu(h @ weight(w["gate"]).T) * (h @ weight(w["up"]).T)) @ weight(w["down"]).T
    return 3.0 * norm(x[:, -1]) @ weight(d.head).T


@pytest.mark.parametrize("B,P,cache", [(1, 5, torch.bfloat16), (3, 40, torch.bfloat16), (16, 3, torch.bfloat16)])
def test_generation_matches_a_dense_recomputation(example, B, P, cache):
    """Activations are rounded to bf16 (2^-8) at about six places per layer and the cache once more; over two layers the
    relative error of the logits' rows (2-norm) stays well below 12 * 2^-8 = 4.7%."""
    new = 6
    d = example.Decoder(B, P + new, cache_dtype=cache)
    prompt = torch.randint(0, d.V, (B, P), generator=torch.Generator().manual_seed(3)).cuda()
    out, logits = d.generate(prompt, new)
    torch.cuda.synchronize()
    assert kq.kq_device_error() == 0
    assert torch.all((out >= 0) & (out < d.V))
    want = dense_logits(d, torch.cat([prompt, out], 1))
    err = (logits.double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(err.max()) < 12 * 2.0 ** -8, err.tolist()
    again, _ = example.Decoder(B, P + new, cache_dtype=cache).generate(prompt, new)
    assert torch.equal(again, out)
