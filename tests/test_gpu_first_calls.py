"""Calls of several threads at once, each kernel's first ones in their process: a kernel's settings are made at its first call,
and have to serve batches of all sizes, whichever thread makes them last."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading
import torch
from gguf_quant_weight_super_gb300 import kq

kq.lib()
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
sizes = [4096, 8, 2600, 16, 1111, 300, 64, 4000]
g = torch.Generator("cuda").manual_seed(1)
tables = {B: torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1) for B in sizes}
lens = {B: torch.full((B,), T, dtype=torch.int32, device="cuda") for B in sizes for T in [4]}
streams = [torch.cuda.Stream() for _ in sizes]
bad = []
for tree in (False, True):
    for q_dtype, dtype, D, G in [(BF16, BF16, 128, 16), (BF16, BF16, 64, 1), (F32, BF16, 64, 4), (BF16, F8, 128, 8), (F32, F8, 256, 2)]:
        k, v = ((torch.randn((4096, 4, 1, D), device="cuda", generator=g) * 3).to(dtype) for _ in range(2))
        cache, jobs = kq.KVCache(k, v), []
        for B in sizes:
            q = torch.randn((B, 4, G, D), device="cuda", generator=g).to(q_dtype)
            mask = torch.tensor([[1, 3, 5, 11]], device="cuda").repeat(B, 1)
            ws = kq.attn_tree_workspace(cache, B, 4, G) if tree else kq.attn_workspace(cache, B, 4, G)
            jobs.append((B, q, mask, ws, torch.empty_like(q)))
        torch.cuda.synchronize()
        start = threading.Barrier(len(jobs))

        def call(i, wait=True):
            B, q, mask, ws, out = jobs[i]
            if wait:
                start.wait()
            try:
                if tree:
                    kq.attn_tree(cache, tables[B], lens[B], mask, q, ws, out=out, stream=streams[i])
                else:
                    kq.attn_decode(cache, tables[B], lens[B], q, ws, out=out, stream=streams[i])
            except kq.KQError as e:
                bad.append((tree, str(q_dtype), str(dtype), D, B, "at once" if wait else "later", str(e)))
        threads = [threading.Thread(target=call, args=(i,)) for i in range(len(jobs))]
        [t.start() for t in threads]
        [t.join() for t in threads]
        torch.cuda.synchronize()
        for i in range(len(jobs)):
            call(i, False)
        torch.cuda.synchronize()
        # the first sequences of the largest batch, in 64 bits
        B, q, mask, ws, out = jobs[0]
        sees = (mask[:, :, None] >> torch.arange(4, device="cuda") & 1).bool() if tree else torch.ones(4, 4, device="cuda").tril().bool()[None]
        s = torch.einsum("bthd,bjd->bhtj", q.double(), k[:, :, 0].double()) * D ** -0.5
        p = torch.softmax(s.masked_fill(~sees[:, None], float("-inf")), -1)
        ref = torch.einsum("bhtj,bjd->bthd", p, v[:, :, 0].double())
        if not bool(((out.double() - ref).abs() <= 2.0 ** -7 * 20).all()):
            bad.append((tree, str(q_dtype), str(dtype), D, "wrong"))
print(bad)
raise SystemExit(1 if bad else 0)
"""


@pytest.mark.gpu
def test_first_calls_of_several_threads_with_batches_of_all_sizes():
    require_gpu()
    from gguf_quant_weight_super_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
