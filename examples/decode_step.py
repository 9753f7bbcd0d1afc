"""Decoding with quantized weights, end to end on the library's calls: for each layer the q|k|v products, kv_append
(norms, rotation, cache), attn_decode, the o product and a gated FFN; after the LM head, sample.  The weights are random
Q4_K blocks, so the text means nothing; torch looks up embeddings, norms the hidden rows and adds.

    python examples/decode_step.py [--sequences 4] [--prompt 37] [--new 16]

Prompts go through in blocks of up to 16 rows (sequences x tokens), as a verify block of drafted tokens would; then one
token of each sequence per step."""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gguf_quant_weight_super_gb300 import kq, synth  # noqa: E402

Q4_K = synth.Q4_K


def random_blocks(n, k, g):
    """An n x k matrix (k a multiple of 256) of Q4_K blocks with weights d (q - 7.5) / sqrt(k), about unit rows: all
    six-bit scales and mins 32, dmin = 7.5 d."""
    b = np.zeros((n * k // 256, 144), np.uint8)
    d = (g.uniform(0.8, 1.2, (len(b), 1)) / (32 * 4.61 * k ** 0.5)).astype(np.float16)
    b[:, :4] = np.concatenate([d, (7.5 * d.astype(np.float32)).astype(np.float16)], 1).view(np.uint8)
    b[:, 4:12] = 0xA0
    b[:, 16:] = g.integers(0, 256, (len(b), 128))
    return torch.from_numpy(b.reshape(-1)).cuda()


class Decoder:
    """A small decoder: weights, one paged cache per layer, and the calls' workspaces."""

    def __init__(self, sequences, positions, layers=2, hidden=512, heads=8, kv_heads=2, head_dim=128, ffn=1024, vocab=4096,
                 page=16, cache_dtype=torch.bfloat16, seed=0):
        g = synth.rng(900, seed)
        self.B, self.H, self.heads, self.kv, self.D, self.F, self.V = sequences, hidden, heads, kv_heads, head_dim, ffn, vocab

        def matrix(n, k):
            return random_blocks(n, k, g), n, k

        q, kvd = heads * head_dim, kv_heads * head_dim
        self.layers = []
        pages = -(-positions // page)
        t = torch.Generator().manual_seed(seed)
        for _ in range(layers):
            k = torch.zeros((sequences * pages, page, kv_heads, head_dim), device="cuda").to(cache_dtype)
            self.layers.append(dict(
                q=matrix(q, hidden), k=matrix(kvd, hidden), v=matrix(kvd, hidden), o=matrix(hidden, q),
                gate=matrix(ffn, hidden), up=matrix(ffn, hidden), down=matrix(hidden, ffn),
                rope=kq.RopeNorm(kq.rope_table(positions, head_dim, base=1e6),
                                 q_norm=(1 + 0.1 * torch.randn(head_dim, generator=t)).cuda(),
                                 k_norm=(1 + 0.1 * torch.randn(head_dim, generator=t)).cuda()),
                cache=kq.KVCache(k, torch.zeros_like(k))))
        self.head = matrix(vocab, hidden)
        self.embedding = torch.randn((vocab, hidden), generator=t).cuda()
        # any order of pages will do
        self.table = torch.randperm(sequences * pages, generator=t).to(torch.int32).view(sequences, pages).cuda()
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.ws = {}

    def norm(self, x):
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def product(self, w, x):
        return kq.matvec(Q4_K, w[0], x, w[1], w[2])

    def step(self, tokens):
        """Logits [B, T, V] after T new tokens of each sequence (tokens [B, T])."""
        B, T = tokens.shape
        D = self.D
        self.lens += T
        x = self.embedding[tokens].view(B * T, self.H)
        for i, w in enumerate(self.layers):
            h = self.norm(x)
            q, k, v = (self.product(w[n], h).view(B, T, -1, D) for n in ("q", "k", "v"))
            q = kq.kv_append(w["cache"], self.table, self.lens, q, k, v, w["rope"])
            if T not in self.ws:
                self.ws[T] = kq.attn_workspace(w["cache"], B, T, self.heads)
            a = kq.attn_decode(w["cache"], self.table, self.lens, q, self.ws[T])
            x = x + self.product(w["o"], a.view(B * T, -1))
            h = self.norm(x)
            f = torch.nn.functional.silu(self.product(w["gate"], h)) * self.product(w["up"], h)
            x = x + self.product(w["down"], f.to(torch.bfloat16))
        return 3.0 * self.product(self.head, self.norm(x)).view(B, T, self.V)

    def generate(self, prompt, new, seed=1, temperature=0.8, top_k=40, top_p=0.95):
        """`new` tokens after prompt [B, P]; returns [B, new] and the last step's logits [B, V]."""
        B, P = prompt.shape
        per = max(1, 16 // B)
        for i in range(0, P, per):
            logits = self.step(prompt[:, i:i + per])[:, -1]
        g = torch.Generator("cuda").manual_seed(seed)
        row = dict(device="cuda", dtype=torch.float32)
        settings = dict(temperature=torch.full((B,), temperature, **row), top_p=torch.full((B,), top_p, **row),
                        top_k=torch.full((B,), top_k, device="cuda", dtype=torch.int32),
                        workspace=kq.sample_workspace(B, self.V))
        out = torch.empty((B, new), dtype=torch.int64, device="cuda")
        for i in range(new):
            ids, _ = kq.sample(logits.contiguous(), torch.rand(B, generator=g, **row), **settings)
            out[:, i] = ids
            logits = self.step(out[:, i:i + 1])[:, -1]
        return out, logits


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=37)
    ap.add_argument("--new", type=int, default=16)
    a = ap.parse_args()
    if not 1 <= a.sequences <= 16:
        ap.error("1 to 16 sequences (the products take up to 16 rows)")
    d = Decoder(a.sequences, a.prompt + a.new)
    prompt = torch.randint(0, d.V, (a.sequences, a.prompt), generator=torch.Generator().manual_seed(2)).cuda()
    out, _ = d.generate(prompt, a.new)
    if kq.kq_device_error():
        raise RuntimeError("device error %d" % kq.kq_device_error())
    for row in out.tolist():
        print(" ".join(str(t) for t in row))


if __name__ == "__main__":
    main()
