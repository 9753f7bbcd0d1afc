"""Thin Python binding of libkq's C ABI (include/kq.h): argument marshalling only.

Every function named ``kq_*`` here calls the C function of the same name with
the device pointers of the given torch tensors and the current CUDA stream;
all computation happens in libkq's CUDA kernels.  There is no fallback: if
libkq.so is missing or fails to load, importing the library raises.
``stream`` (a torch stream or a handle) in place of the current one: the caller
orders and keeps the tensors it passes; those that the call makes itself are
made on that stream.
"""
from __future__ import annotations

import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkq.so")

KQ_Q4_K, KQ_Q5_K, KQ_Q6_K, KQ_IA4 = 1, 2, 3, 4
KQ_F32, KQ_BF16, KQ_F8E4M3 = 0, 1, 2
KQ_ACT_SILU, KQ_ACT_GELU_TANH = 0, 1
KQ_OK = 0
STATUS = {0: "KQ_OK", -1: "KQ_ERR_ARG", -2: "KQ_ERR_TYPE", -3: "KQ_ERR_SHAPE", -4: "KQ_ERR_UNSUPPORTED",
          -5: "KQ_ERR_ALIGN", -6: "KQ_ERR_CUDA", -7: "KQ_ERR_WORKSPACE", -8: "KQ_ERR_DEVICE"}

# exported symbols and their C signatures (kept in step with include/kq.h)
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "kq_block_bytes": (_SZ, [_I]),
    "kq_ia4_pack": (_I, [_P, _P, _P, _I64, _I64, _P, _P]),
    "kq_unpack": (_I, [_I, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "kq_dequant": (_I, [_I, _P, _P, _I64, _P]),
    "kq_dequant_bf16": (_I, [_I, _P, _P, _I64, _P]),
    "kq_moe_route": (_I, [_P, _I64, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _SZ, _P]),
    "kq_matvec": (_I, [_I, _P, _P, _I, _P, _I64, _I64, _I64, _P]),
    "kq_chain_workspace_size": (_SZ, [_P, _I]),
    "kq_chain_prepare": (_I, [_P, _I, _P, _SZ, _P, _P]),
    "kq_chain_run": (_I, [_P, _P, _P]),
    "kq_moe_workspace_size": (_SZ, [_I64, _I64, ctypes.c_int32, ctypes.c_int32]),
    "kq_moe_matvec": (_I, [_I, _P, ctypes.c_int32, _P, _P, _P, _I, _I, _P, _I64, _I64, _I64, ctypes.c_int32,
                           _P, _SZ, _P]),
    "kq_moe_check": (_I, [_P, _P]),
    "kq_selftest_wait": (_I, [_I, ctypes.POINTER(ctypes.c_int), _P]),
    "kq_moe_ffn_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, ctypes.c_int32, ctypes.c_int32]),
    "kq_moe_ffn_offsets": (_I, [_I64, _I64, _I64, _I64, ctypes.c_int32, ctypes.c_int32,
                                ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "kq_moe_ffn": (_I, [_P, _P, _P, _P, _I, _P, _I64, _I64, ctypes.c_int32, _P, _SZ, _P]),
    "kq_moe_matvec_noalloc": (_I, [_I, _P, ctypes.c_int32, _P, _P, _P, _I, _I, _P, _I64, _I64, _I64,
                                   ctypes.c_int32, _P]),
    "kq_kv_append": (_I, [_P, _P, _I64, _P, _I64, _I64, _P, _P, _P, _I, _I64, _I64, _I64, ctypes.c_int32, _P, _P, _I,
                          _P]),
    "kq_attn_workspace_size": (_SZ, [_P, _I64, _I64, ctypes.c_int32]),
    "kq_attn_decode": (_I, [_P, _P, _I64, _P, _I64, _I64, _P, _I, _I64, ctypes.c_int32, ctypes.c_float,
                            ctypes.c_float, ctypes.c_int32, _P, _P, _SZ, _P]),
    "kq_selftest_attn_ctas": (_I, [_P, _I64, _I64, _I, ctypes.c_int32, ctypes.POINTER(ctypes.c_int),
                                   ctypes.POINTER(ctypes.c_int)]),
    "kq_kv_append_tree": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P, _I, _I64, _I64, _I64, ctypes.c_int32, _P, _P,
                               _I, _P]),
    "kq_attn_tree_workspace_size": (_SZ, [_P, _I64, _I64, ctypes.c_int32]),
    "kq_attn_tree": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _I, _I64, ctypes.c_int32, ctypes.c_float, ctypes.c_float,
                          ctypes.c_int32, _P, _P, _SZ, _P]),
    "kq_tree_accept": (_I, [_P, ctypes.c_int32, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    "kq_latent_accept": (_I, [_P, ctypes.c_int32, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    "kq_latent_append": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _I64, ctypes.c_int32, _P,
                              _P, _P]),
    "kq_latent_attn_workspace_size": (_SZ, [_P, _I64, _I64, ctypes.c_int32]),
    "kq_latent_attn": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _I64, ctypes.c_int32, ctypes.c_float, _P, _P, _SZ, _P]),
    "kq_sample_workspace_size": (_SZ, [_I64, _I64]),
    "kq_sample": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "kq_device_error": (_I, [ctypes.POINTER(ctypes.c_int), _I]),
    "kq_last_cuda_error": (_I, []),
    "kq_status_string": (ctypes.c_char_p, [_I]),
}


# The sources each kernel family is compiled from (the one-token / program
# kernel: kq_gemv_kernel.cuh, the translation units that instantiate it and
# the headers it includes).
KERNEL_SOURCES = {
    "prog_kernel": ("kq_gemv_kernel.cuh", "kq_gemv.cu", "kq_gemv_q4k.cu", "kq_gemv_q5k.cu", "kq_gemv_q6k.cu",
                    "kq_gemv_ia4.cu", "kq_lane.cuh", "kq_ptx.cuh", "kq_internal.h", "kq_decode.cuh"),
}


def build_id(kernel=None) -> str:
    """Hash of the kernel sources (identifies which code a profile was taken
    on): all of csrc, or only the files of one kernel family."""
    import glob
    import hashlib
    h = hashlib.sha256()
    if kernel is None:
        files = sorted(glob.glob(os.path.join(PKG, "csrc", "*")))
    else:
        files = [os.path.join(PKG, "csrc", n) for n in KERNEL_SOURCES[kernel]]
    for f in files:
        with open(f, "rb") as fh:
            h.update(os.path.basename(f).encode())
            h.update(fh.read())
    return h.hexdigest()[:16]


class KQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _lib.kq_status_string(status).decode() if _lib is not None else ""
        extra = ""
        if status == -6 and _lib is not None:
            extra = f" (cudaError {_lib.kq_last_cuda_error()})"
        super().__init__(f"{fn}: {STATUS.get(status, status)} -- {msg}{extra}")


_lib = None


def use_timeline_library() -> ctypes.CDLL:
    """Build and load libkq_timeline.so (the library with the one-token
    kernel's per-CTA timer stamps) in place of libkq.so; call before any other
    use of the library in the process."""
    global LIB_PATH
    if _lib is not None:
        raise RuntimeError("the library is already loaded")
    from . import build
    LIB_PATH = build.build(timeline=True)
    L = lib()
    L.kq_timeline_read.restype = ctypes.c_int
    L.kq_timeline_read.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    return L


def lib() -> ctypes.CDLL:
    """Load libkq.so (built in-tree by ``gguf_quant_weight_super_gb300.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libkq.so not built ({LIB_PATH}); run gguf_quant_weight_super_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libkq takes device tensors only")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        if torch.cuda.is_initialized():  # the current stream's handle without a Stream object around it
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _new(stream, make, *args, **kw):
    """make(...), a tensor of the call's own: made on the stream that the call runs on, so that its memory is neither written
    by earlier work of another stream nor handed on while the call's kernels use it."""
    if stream is None:
        return make(*args, **kw)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _check(fn: str, status: int):
    if status != KQ_OK:
        raise KQError(fn, status)


def kq_block_bytes(qtype: int) -> int:
    return lib().kq_block_bytes(qtype)


def kq_unpack(qtype, blocks, n_blocks, codes=None, scales=None, mins=None, d_bits=None, dmin_bits=None,
              stream=None):
    _check("kq_unpack", lib().kq_unpack(qtype, _ptr(blocks), n_blocks, _ptr(codes), _ptr(scales), _ptr(mins),
                                        _ptr(d_bits), _ptr(dmin_bits), _stream(stream)))


def kq_dequant(qtype, blocks, out, n, stream=None):
    _check("kq_dequant", lib().kq_dequant(qtype, _ptr(blocks), _ptr(out), n, _stream(stream)))


def kq_moe_route(logits, M, n_experts, top_k, expert_ids, gate_w, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("kq_moe_route", lib().kq_moe_route(_ptr(logits), M, n_experts, top_k, _ptr(expert_ids), _ptr(gate_w),
                                              _ptr(workspace), ws_bytes, _stream(stream)))


def moe_route(logits: torch.Tensor, top_k: int, workspace=None, stream=None):
    """(ids int32 [M, top_k], gate fp32 [M, top_k]) for logits [M, n_experts] (kq_moe_route)."""
    M, E = logits.shape
    ids = _new(stream, torch.empty, (M, top_k), dtype=torch.int32, device=logits.device)
    gate = _new(stream, torch.empty, (M, top_k), dtype=torch.float32, device=logits.device)
    kq_moe_route(logits, M, E, top_k, ids, gate, workspace, stream)
    return ids, gate


def kq_ia4_pack(q, scales, biases, N, K, blocks, stream=None):
    _check("kq_ia4_pack", lib().kq_ia4_pack(_ptr(q), _ptr(scales), _ptr(biases), N, K, _ptr(blocks),
                                            _stream(stream)))


def ia4_pack(q: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor) -> torch.Tensor:
    """MLX group-affine INT4 arrays (int32 codes [N, K/8], bf16-bit scales and
    biases [N, K/64] as int16 or bfloat16) -> KQ_IA4 blocks (uint8)."""
    N, K = q.shape[0], q.shape[1] * 8
    out = torch.empty(N * ((K + 255) // 256) * 144, dtype=torch.uint8, device=q.device)
    kq_ia4_pack(q, scales, biases, N, K, out)
    return out


def kq_dequant_bf16(qtype, blocks, out, n, stream=None):
    _check("kq_dequant_bf16", lib().kq_dequant_bf16(qtype, _ptr(blocks), _ptr(out), n, _stream(stream)))


def kq_matvec(qtype, W, x, x_dtype, y, N, K, M, stream=None):
    _check("kq_matvec", lib().kq_matvec(qtype, _ptr(W), _ptr(x), x_dtype, _ptr(y), N, K, M, _stream(stream)))


class KqOp(ctypes.Structure):
    """struct kq_op of include/kq.h."""
    _fields_ = [("type", ctypes.c_int32), ("x_dtype", ctypes.c_int32), ("wait_previous", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("W", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class KqChainPlan(ctypes.Structure):
    """struct kq_chain_plan of include/kq.h (opaque)."""
    _fields_ = [("opaque", ctypes.c_int64 * 8)]


def _op_array(ops):
    arr = (KqOp * len(ops))()
    for i, o in enumerate(ops):
        arr[i] = KqOp(o["type"], o["x_dtype"], int(o.get("wait_previous", 0)), 0, _ptr(o["W"]), _ptr(o["x"]),
                      _ptr(o["y"]), o["N"], o["K"])
    return arr


def kq_chain_workspace_size(ops) -> int:
    arr = _op_array(ops)
    return lib().kq_chain_workspace_size(ctypes.cast(arr, ctypes.c_void_p), len(ops))


def kq_chain_prepare(ops, workspace, workspace_bytes, plan: KqChainPlan, stream=None):
    arr = _op_array(ops)
    _check("kq_chain_prepare", lib().kq_chain_prepare(ctypes.cast(arr, ctypes.c_void_p), len(ops), _ptr(workspace),
                                                      workspace_bytes, ctypes.cast(ctypes.pointer(plan), ctypes.c_void_p),
                                                      _stream(stream)))


def kq_chain_run(plan: KqChainPlan, workspace, stream=None):
    _check("kq_chain_run", lib().kq_chain_run(ctypes.cast(ctypes.pointer(plan), ctypes.c_void_p), _ptr(workspace),
                                              _stream(stream)))


def kq_moe_workspace_size(N, M, top_k, n_experts) -> int:
    return lib().kq_moe_workspace_size(N, M, top_k, n_experts)


def kq_moe_matvec(qtype, W_experts, n_experts, expert_ids, gate_w, x, x_dtype, x_per_slot, y, N, K, M, top_k,
                  workspace, workspace_bytes, stream=None):
    _check("kq_moe_matvec", lib().kq_moe_matvec(qtype, _ptr(W_experts), n_experts, _ptr(expert_ids), _ptr(gate_w),
                                                _ptr(x), x_dtype, int(x_per_slot), _ptr(y), N, K, M, top_k,
                                                _ptr(workspace), workspace_bytes, _stream(stream)))


def kq_moe_matvec_noalloc(qtype, W_experts, n_experts, expert_ids, gate_w, x, x_dtype, x_per_slot, y, N, K, M,
                          top_k, stream=None):
    _check("kq_moe_matvec_noalloc",
           lib().kq_moe_matvec_noalloc(qtype, _ptr(W_experts), n_experts, _ptr(expert_ids), _ptr(gate_w), _ptr(x),
                                       x_dtype, int(x_per_slot), _ptr(y), N, K, M, top_k, _stream(stream)))


def kq_moe_check(workspace, stream=None):
    _check("kq_moe_check", lib().kq_moe_check(_ptr(workspace), _stream(stream)))


def moe_workspace(N, M, top_k, n_experts, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor for kq_moe_matvec (the caching allocator aligns it to 512 bytes)."""
    n = kq_moe_workspace_size(N, M, top_k, n_experts)
    if n == 0:
        raise KQError("kq_moe_workspace_size", -4)
    return torch.zeros(n, dtype=torch.uint8, device=device)


class KqMoeFfnWeights(ctypes.Structure):
    """struct kq_moe_ffn_weights of include/kq.h."""
    _fields_ = [("type_gate_up", ctypes.c_int32), ("type_down", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("act", ctypes.c_int32), ("F", ctypes.c_int64), ("SH", ctypes.c_int64),
                ("W_gate", ctypes.c_void_p), ("W_up", ctypes.c_void_p), ("W_down", ctypes.c_void_p),
                ("Ws_gate", ctypes.c_void_p), ("Ws_up", ctypes.c_void_p), ("Ws_down", ctypes.c_void_p)]


def ffn_weights(type_gate_up, type_down, n_experts, act, F, W_gate, W_up, W_down, SH=0, Ws_gate=None, Ws_up=None,
                Ws_down=None) -> KqMoeFfnWeights:
    return KqMoeFfnWeights(type_gate_up, type_down, n_experts, act, F, SH, _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                           _ptr(Ws_gate), _ptr(Ws_up), _ptr(Ws_down))


def kq_moe_ffn_workspace_size(H, F, SH, M, top_k, n_experts) -> int:
    return lib().kq_moe_ffn_workspace_size(H, F, SH, M, top_k, n_experts)


def kq_moe_ffn_offsets(H, F, SH, M, top_k, n_experts):
    """(byte offset of h [M*top_k][F], byte offset of hs [M][SH]) in the workspace."""
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("kq_moe_ffn_offsets", lib().kq_moe_ffn_offsets(H, F, SH, M, top_k, n_experts, ctypes.byref(a),
                                                          ctypes.byref(b)))
    return a.value, b.value


def moe_ffn_workspace(H, F, SH, M, top_k, n_experts, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor for kq_moe_ffn."""
    n = kq_moe_ffn_workspace_size(H, F, SH, M, top_k, n_experts)
    if n == 0:
        raise KQError("kq_moe_ffn_workspace_size", -4)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kq_moe_ffn(weights: KqMoeFfnWeights, expert_ids, gate_w, x, x_dtype, y, H, M, top_k, workspace,
               workspace_bytes, stream=None):
    _check("kq_moe_ffn", lib().kq_moe_ffn(ctypes.cast(ctypes.pointer(weights), ctypes.c_void_p), _ptr(expert_ids),
                                          _ptr(gate_w), _ptr(x), x_dtype, _ptr(y), H, M, top_k, _ptr(workspace),
                                          workspace_bytes, _stream(stream)))


def kq_selftest_wait(kind: int, stream=None) -> int:
    """Run the bounded-wait self-test (0: mbarrier, 1: grid barrier); returns the observed error code."""
    code = ctypes.c_int(-1)
    _check("kq_selftest_wait", lib().kq_selftest_wait(kind, ctypes.byref(code), _stream(stream)))
    return code.value


def kq_device_error(clear: bool = False) -> int:
    code = ctypes.c_int(0)
    st = lib().kq_device_error(ctypes.byref(code), int(clear))
    if st not in (KQ_OK, -8):
        raise KQError("kq_device_error", st)
    return code.value


# ---------------------------------------------------------------------------
# Convenience wrappers that allocate outputs with torch (still one C call each).
# ---------------------------------------------------------------------------

def x_dtype_of(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return KQ_F32
    if x.dtype == torch.bfloat16:
        return KQ_BF16
    raise TypeError("x must be float32 or bfloat16")


def matvec(qtype: int, W: torch.Tensor, x: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None):
    """y = W x for x of shape (M, K) (or (K,)); returns fp32 (M, N)."""
    x2 = x.reshape(-1, K)
    M = x2.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
    kq_matvec(qtype, W, x2, x_dtype_of(x2), y, N, K, M)
    return y


class Chain:
    """A prepared chain of one-token products (kq_chain_* of include/kq.h).

    ops: dicts with keys type, x_dtype, W, x, y, N, K and optionally
    wait_previous; the tensors must stay alive while the chain is used.
    The workspace is a torch uint8 tensor owned by this object.
    """

    def __init__(self, ops, device=None, stream=None):
        self.ops = list(ops)
        n = kq_chain_workspace_size(self.ops)
        if n == 0:
            raise KQError("kq_chain_workspace_size", -4)
        dev = device if device is not None else self.ops[0]["y"].device
        self.workspace = _new(stream, torch.empty, n + 256, dtype=torch.uint8, device=dev)
        off = (-self.workspace.data_ptr()) % 256
        self._ws_ptr = self.workspace.data_ptr() + off
        self._ws_bytes = n
        self.plan = KqChainPlan()
        kq_chain_prepare(self.ops, self._ws_ptr, self._ws_bytes, self.plan, stream)

    def run(self, stream=None):
        kq_chain_run(self.plan, self._ws_ptr, stream)


def dequant(qtype: int, blocks: torch.Tensor, n: int) -> torch.Tensor:
    out = torch.empty(n, dtype=torch.float32, device=blocks.device)
    kq_dequant(qtype, blocks, out, n)
    return out


def dequant_bf16(qtype: int, blocks: torch.Tensor, n: int) -> torch.Tensor:
    """The weights as a torch.bfloat16 tensor (kq_dequant_bf16)."""
    out = torch.empty(n, dtype=torch.bfloat16, device=blocks.device)
    kq_dequant_bf16(qtype, blocks, out, n)
    return out


# ---------------------------------------------------------------------------
# The paged key-value cache, its writer and its reader, and the sampler.
# ---------------------------------------------------------------------------

class KqKvCache(ctypes.Structure):
    """struct kq_kv_cache of include/kq.h."""
    _fields_ = [("dtype", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class KqRope(ctypes.Structure):
    """struct kq_rope of include/kq.h."""
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("norm_offset", ctypes.c_float), ("cos_sin", ctypes.c_void_p), ("n_positions", ctypes.c_int64),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


_CACHE_TYPES = {torch.bfloat16: KQ_BF16, torch.float8_e4m3fn: KQ_F8E4M3}


class KVCache:
    """A layer's cache: k and v [n_pages, page_size, n_kv_heads, head_dim], bfloat16 or float8_e4m3fn (stored values
    times k_scale, v_scale), of any strides but a contiguous last dimension (a permuted view gives another order of
    slots and heads).  Holds both tensors."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v: alike, [n_pages, page_size, n_kv_heads, head_dim], last dimension contiguous")
        if k.dtype not in _CACHE_TYPES:
            raise TypeError("a cache is bfloat16 or float8_e4m3fn")
        self.k, self.v, self.k_scale, self.v_scale = k, v, float(k_scale), float(v_scale)
        n_pages, page, heads, dim = k.shape
        self.struct = KqKvCache(_CACHE_TYPES[k.dtype], heads, dim, page, n_pages, k.stride(0), k.stride(1), k.stride(2),
                                _ptr(k), _ptr(v), self.k_scale, self.v_scale)
        self._ref = ctypes.addressof(self.struct)
        self.n_kv_heads, self.head_dim = heads, dim


class RopeNorm:
    """What kv_append does to q and k (struct kq_rope): norm weights [head_dim] fp32 or None, and cos_sin
    [n_positions, rot_dim] fp32 (see rope_table) or None for no rotation.  Holds the tensors."""

    def __init__(self, cos_sin=None, interleaved: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6,
                 norm_offset: float = 0.0):
        for w in (cos_sin, q_norm, k_norm):
            if w is not None and (w.dtype != torch.float32 or not w.is_contiguous()):
                raise TypeError("cos_sin, q_norm and k_norm are contiguous float32")
        self.cos_sin, self.q_norm, self.k_norm = cos_sin, q_norm, k_norm
        n, rot = cos_sin.shape if cos_sin is not None else (0, 0)
        self.struct = KqRope(_ptr(q_norm), _ptr(k_norm), eps, norm_offset, _ptr(cos_sin), n, rot, int(interleaved))
        self._ref = ctypes.addressof(self.struct)
        dims = {w.numel() for w in (q_norm, k_norm) if w is not None}
        if len(dims) > 1:
            raise ValueError("norm weights: [head_dim]")
        self.norm_dim = dims.pop() if dims else 0


def rope_table(n_positions: int, rot_dim: int, base: float = 10000.0, factor: float = 1.0, trained: int = 0,
               low: float = 1.0, high: float = 4.0, amplitude: float = 1.0, device="cuda") -> torch.Tensor:
    """cos | sin [n_positions, rot_dim] fp32 for RopeNorm, computed in 64 bits: pair i turns by base^(-2i/rot_dim) per
    position.  factor > 1 stretches positions: all pairs alike (trained = 0), or, given the context length the model
    was trained on, the pairs that turn at most `low` times over it, none that turn at least `high` times, and a
    linear blend between.  amplitude multiplies the table."""
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    if factor != 1.0:
        keep = torch.zeros_like(freq)
        if trained:
            turns = trained * freq / (2 * torch.pi)
            keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    a = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * freq
    return (torch.cat([a.cos(), a.sin()], 1) * amplitude).float()


def kq_kv_append(cache, page_table, max_pages, seq_lens, B, T, q, k, v, x_dtype, q_stride, k_stride, v_stride, n_q_heads,
                 rope, q_out, q_out_dtype, stream=None):
    _check("kq_kv_append", lib().kq_kv_append(cache, _ptr(page_table), max_pages, _ptr(seq_lens), B, T, _ptr(q), _ptr(k),
                                              _ptr(v), x_dtype, q_stride, k_stride, v_stride, n_q_heads, rope,
                                              _ptr(q_out), q_out_dtype, _stream(stream)))


def kq_attn_workspace_size(cache, B, T, n_q_heads) -> int:
    return lib().kq_attn_workspace_size(cache, B, T, n_q_heads)


def kq_attn_decode(cache, page_table, max_pages, seq_lens, B, T, q, q_dtype, q_stride, n_q_heads, scale, softcap, window,
                   out, workspace, workspace_bytes, stream=None):
    _check("kq_attn_decode", lib().kq_attn_decode(cache, _ptr(page_table), max_pages, _ptr(seq_lens), B, T, _ptr(q),
                                                  q_dtype, q_stride, n_q_heads, scale, softcap, window, _ptr(out),
                                                  _ptr(workspace), workspace_bytes, _stream(stream)))


def kq_selftest_attn_ctas(cache, B, T, q_dtype, n_q_heads):
    """(planned, resident) CTAs per SM of an attention call."""
    n = ctypes.c_int(0), ctypes.c_int(0)
    _check("kq_selftest_attn_ctas", lib().kq_selftest_attn_ctas(cache, B, T, q_dtype, n_q_heads, *map(ctypes.byref, n)))
    return n[0].value, n[1].value


def kq_sample_workspace_size(M, V) -> int:
    return lib().kq_sample_workspace_size(M, V)


def kq_sample(logits, dtype, row_stride, M, V, u, temperature, top_k, top_p, min_p, ids, probs, workspace,
              workspace_bytes, stream=None):
    _check("kq_sample", lib().kq_sample(_ptr(logits), dtype, row_stride, M, V, _ptr(u), _ptr(temperature), _ptr(top_k),
                                        _ptr(top_p), _ptr(min_p), _ptr(ids), _ptr(probs), _ptr(workspace),
                                        workspace_bytes, _stream(stream)))


# The calls below are made once per layer and token, where a Python call's own time counts: each property of a tensor is
# looked up once, in line.

_DTYPE_CODE = {torch.float32: KQ_F32, torch.bfloat16: KQ_BF16}
_f32, _i32, _i64, _u8 = torch.float32, torch.int32, torch.int64, torch.uint8


def _row_stride(name: str, x: torch.Tensor, B: int, T: int, heads: int, D: int) -> int:
    """The row stride of x [B, T, heads, D]: heads contiguous, rows at one stride."""
    s0, s1, s2, s3 = x.stride()
    if s3 != 1 or (s2 != D and heads > 1) or (s0 != T * s1 and B > 1 and T > 1):
        raise ValueError(f"{name}: heads contiguous, tokens at one stride")
    return s1 if T > 1 else s0 if B > 1 else heads * D


def _rows(name: str, x: torch.Tensor, B: int, T: int, D: int):
    """The heads and the row stride of x [B, T, heads, D]."""
    shape = x.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != T or shape[3] != D:
        raise ValueError(f"{name}: [{B}, {T}, heads, {D}], not {list(shape)}")
    return shape[2], _row_stride(name, x, B, T, shape[2], D)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent from builds without CUDA, as _cuda_getDevice
_device = getattr(torch._C, "_cuda_getDevice", None)


def _host():
    return ValueError("libkq takes device tensors only")


def _here():
    """The current device's current stream (a device tensor is at hand, so CUDA is up)."""
    return _raw_stream(_device())


def kv_append(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
              v: torch.Tensor, rope: RopeNorm, q_out: torch.Tensor | None = None, q_out_dtype=torch.bfloat16,
              stream=None) -> torch.Tensor:
    """kq_kv_append for q [B, T, n_q_heads, head_dim], k and v [B, T, n_kv_heads, head_dim] (views of one fused buffer
    will do), page_table [B, max_pages] and seq_lens [B] int32; returns q_out."""
    shape, kv_shape, D, heads, dtype = q.shape, k.shape, cache.head_dim, cache.n_kv_heads, q.dtype
    if len(shape) != 4 or shape[3] != D:
        raise ValueError(f"q: [B, T, heads, {D}], not {list(shape)}")
    B, T, Hq, _ = shape
    if kv_shape != (B, T, heads, D) or v.shape != kv_shape or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError(f"k and v: [{B}, {T}, {heads}, {D}], of q's type")
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("q, k and v are float32 or bfloat16")
    if rope.norm_dim != 0 and rope.norm_dim != D:
        raise ValueError("norm weights: [head_dim]")
    if q_out is None:
        q_out = _new(stream, torch.empty, shape, dtype=q_out_dtype, device=q.device)
    elif q_out.shape != shape or not q_out.is_contiguous():
        raise ValueError("q_out: contiguous, of q's shape")
    out_code = _DTYPE_CODE.get(q_out.dtype)
    if out_code is None:
        raise TypeError("q_out is float32 or bfloat16")
    rows, W = page_table.shape
    if page_table.dtype is not _i32 or rows != B or not page_table.is_contiguous():
        raise ValueError(f"page_table: contiguous int32 [{B}, max_pages]")
    if seq_lens.dtype is not _i32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens: contiguous int32 [{B}]")
    if not (q.is_cuda and k.is_cuda and v.is_cuda and q_out.is_cuda and page_table.is_cuda and seq_lens.is_cuda):
        raise _host()
    status = (_lib or lib()).kq_kv_append(
        cache._ref, page_table.data_ptr(), W, seq_lens.data_ptr(), B, T, q.data_ptr(), k.data_ptr(), v.data_ptr(), code,
        Hq * D if q.is_contiguous() else _row_stride("q", q, B, T, Hq, D),
        heads * D if k.is_contiguous() else _row_stride("k", k, B, T, heads, D),
        heads * D if v.is_contiguous() else _row_stride("v", v, B, T, heads, D), Hq,
        rope._ref, q_out.data_ptr(), out_code, _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_kv_append", status)
    return q_out


def attn_workspace(cache: KVCache, B: int, T: int, n_q_heads: int) -> torch.Tensor:
    """A zero-filled workspace tensor for attn_decode."""
    n = kq_attn_workspace_size(cache._ref, B, T, n_q_heads)
    if n == 0:
        raise KQError("kq_attn_workspace_size", -4)
    return torch.zeros(n, dtype=torch.uint8, device=cache.k.device)


def attn_decode(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, q: torch.Tensor,
                workspace: torch.Tensor, scale: float | None = None, softcap: float = 0.0, window: int = 0,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kq_attn_decode for q [B, T, n_q_heads, head_dim]; scale None: head_dim^-0.5.  Returns out, of q's type."""
    shape, D, dtype = q.shape, cache.head_dim, q.dtype
    if len(shape) != 4 or shape[3] != D:
        raise ValueError(f"q: [B, T, heads, {D}], not {list(shape)}")
    B, T, Hq, _ = shape
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("q is float32 or bfloat16")
    if out is None:
        out = _new(stream, torch.empty, shape, dtype=dtype, device=q.device)
    elif out.shape != shape or out.dtype is not dtype or not out.is_contiguous():
        raise ValueError("out: contiguous, of q's shape and type")
    rows, W = page_table.shape
    if page_table.dtype is not _i32 or rows != B or not page_table.is_contiguous():
        raise ValueError(f"page_table: contiguous int32 [{B}, max_pages]")
    if seq_lens.dtype is not _i32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens: contiguous int32 [{B}]")
    if workspace.dtype is not _u8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8")
    if not (q.is_cuda and out.is_cuda and page_table.is_cuda and seq_lens.is_cuda and workspace.is_cuda):
        raise _host()
    status = (_lib or lib()).kq_attn_decode(
        cache._ref, page_table.data_ptr(), W, seq_lens.data_ptr(), B, T, q.data_ptr(), code,
        Hq * D if q.is_contiguous() else _row_stride("q", q, B, T, Hq, D), Hq, D ** -0.5 if scale is None else scale, softcap, window, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_attn_decode", status)
    return out


# ---- trees of drafted tokens, and latent caches

def kq_kv_append_tree(cache, page_table, max_pages, seq_lens, tree, B, T, q, k, v, x_dtype, q_stride, k_stride, v_stride,
                      n_q_heads, rope, q_out, q_out_dtype, stream=None):
    _check("kq_kv_append_tree", lib().kq_kv_append_tree(cache, _ptr(page_table), max_pages, _ptr(seq_lens), _ptr(tree), B, T,
                                                        _ptr(q), _ptr(k), _ptr(v), x_dtype, q_stride, k_stride, v_stride,
                                                        n_q_heads, rope, _ptr(q_out), q_out_dtype, _stream(stream)))


def kq_attn_tree_workspace_size(cache, B, T, n_q_heads) -> int:
    return lib().kq_attn_tree_workspace_size(cache, B, T, n_q_heads)


def kq_attn_tree(cache, page_table, max_pages, seq_lens, tree, B, T, q, q_dtype, q_stride, n_q_heads, scale, softcap, window,
                 out, workspace, workspace_bytes, stream=None):
    _check("kq_attn_tree", lib().kq_attn_tree(cache, _ptr(page_table), max_pages, _ptr(seq_lens), _ptr(tree), B, T, _ptr(q),
                                              q_dtype, q_stride, n_q_heads, scale, softcap, window, _ptr(out),
                                              _ptr(workspace), workspace_bytes, _stream(stream)))


def kq_tree_accept(caches, n_caches, page_table, max_pages, seq_lens, tree, tokens, ids, B, T, path, count, next_ids, new_lens,
                   stream=None):
    _check("kq_tree_accept", lib().kq_tree_accept(caches, n_caches, _ptr(page_table), max_pages, _ptr(seq_lens), _ptr(tree),
                                                  _ptr(tokens), _ptr(ids), B, T, _ptr(path), _ptr(count), _ptr(next_ids),
                                                  _ptr(new_lens), _stream(stream)))


def kq_latent_accept(caches, n_caches, page_table, max_pages, seq_lens, tree, tokens, ids, B, T, path, count, next_ids,
                     new_lens, stream=None):
    _check("kq_latent_accept", lib().kq_latent_accept(caches, n_caches, _ptr(page_table), max_pages, _ptr(seq_lens),
                                                      _ptr(tree), _ptr(tokens), _ptr(ids), B, T, _ptr(path), _ptr(count),
                                                      _ptr(next_ids), _ptr(new_lens), _stream(stream)))


def kq_latent_append(cache, page_table, max_pages, seq_lens, tree, B, T, q_latent, q_rope, c, x_dtype, q_latent_stride,
                     q_rope_stride, q_rope_head_stride, c_stride, n_heads, rope, q_out, stream=None):
    _check("kq_latent_append", lib().kq_latent_append(cache, _ptr(page_table), max_pages, _ptr(seq_lens), _ptr(tree), B, T,
                                                      _ptr(q_latent), _ptr(q_rope), _ptr(c), x_dtype, q_latent_stride,
                                                      q_rope_stride, q_rope_head_stride, c_stride, n_heads, rope,
                                                      _ptr(q_out), _stream(stream)))


def kq_latent_attn_workspace_size(cache, B, T, n_heads) -> int:
    return lib().kq_latent_attn_workspace_size(cache, B, T, n_heads)


def kq_latent_attn(cache, page_table, max_pages, seq_lens, tree, B, T, q, q_stride, n_heads, scale, out, workspace,
                   workspace_bytes, stream=None):
    _check("kq_latent_attn", lib().kq_latent_attn(cache, _ptr(page_table), max_pages, _ptr(seq_lens), _ptr(tree), B, T,
                                                  _ptr(q), q_stride, n_heads, scale, _ptr(out), _ptr(workspace),
                                                  workspace_bytes, _stream(stream)))


class KqLatentCache(ctypes.Structure):
    """struct kq_latent_cache of include/kq.h."""
    _fields_ = [("dtype", ctypes.c_int32), ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("c", ctypes.c_void_p), ("scale", ctypes.c_float)]


class LatentCache:
    """A layer's latent cache: c [n_pages, page_size, latent_dim + rope_dim], bfloat16 or float8_e4m3fn (stored values times
    scale), of any strides but a contiguous last dimension.  Holds the tensor."""

    def __init__(self, c: torch.Tensor, latent_dim: int, scale: float = 1.0):
        if c.dim() != 3 or c.stride(2) != 1 or not 0 < latent_dim < c.shape[2]:
            raise ValueError("c: [n_pages, page_size, latent_dim + rope_dim], last dimension contiguous")
        if c.dtype not in _CACHE_TYPES:
            raise TypeError("a cache is bfloat16 or float8_e4m3fn")
        self.c, self.scale = c, float(scale)
        self.latent_dim, self.rope_dim = latent_dim, c.shape[2] - latent_dim
        self.struct = KqLatentCache(_CACHE_TYPES[c.dtype], latent_dim, self.rope_dim, c.shape[1], c.shape[0], c.stride(0),
                                    c.stride(1), _ptr(c), self.scale)
        self._ref = ctypes.addressof(self.struct)


class CacheSet:
    """The caches of all layers, all KVCache or all LatentCache, for tree_accept.  Holds them."""

    def __init__(self, caches):
        self.caches = list(caches)
        kinds = {type(c) for c in self.caches}
        if len(kinds) > 1 or not kinds <= {KVCache, LatentCache}:
            raise TypeError("caches are all KVCache or all LatentCache")
        self.latent = kinds == {LatentCache}
        kind = KqLatentCache if self.latent else KqKvCache
        self._array = (kind * len(self.caches))(*(c.struct for c in self.caches))
        self._ref, self.n = (ctypes.addressof(self._array) if self.caches else None), len(self.caches)


def _tables(page_table, seq_lens, tree, B, T):
    """Checks the tensors that say where a call's tokens are; whether all are device tensors, and the table's width."""
    rows, W = page_table.shape
    if page_table.dtype is not _i32 or rows != B or not page_table.is_contiguous():
        raise ValueError(f"page_table: contiguous int32 [{B}, max_pages]")
    if seq_lens.dtype is not _i32 or seq_lens.shape != (B,) or not seq_lens.is_contiguous():
        raise ValueError(f"seq_lens: contiguous int32 [{B}]")
    if tree is not None and (tree.dtype is not _i64 or tree.shape != (B, T) or not tree.is_contiguous()):
        raise ValueError(f"tree: contiguous int64 [{B}, {T}]")
    return page_table.is_cuda and seq_lens.is_cuda and (tree is None or tree.is_cuda), W


def kv_append_tree(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, tree: torch.Tensor, q: torch.Tensor,
                   k: torch.Tensor, v: torch.Tensor, rope: RopeNorm, q_out: torch.Tensor | None = None,
                   q_out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """kv_append of drafted tokens that form a tree (kq_kv_append_tree): tree [B, T] int64, bit u of a token's mask: it sees
    drafted token u."""
    shape, kv_shape, D, heads, dtype = q.shape, k.shape, cache.head_dim, cache.n_kv_heads, q.dtype
    if len(shape) != 4 or shape[3] != D:
        raise ValueError(f"q: [B, T, heads, {D}], not {list(shape)}")
    B, T, Hq, _ = shape
    if kv_shape != (B, T, heads, D) or v.shape != kv_shape or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError(f"k and v: [{B}, {T}, {heads}, {D}], of q's type")
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("q, k and v are float32 or bfloat16")
    if rope.norm_dim != 0 and rope.norm_dim != D:
        raise ValueError("norm weights: [head_dim]")
    if q_out is None:
        q_out = _new(stream, torch.empty, shape, dtype=q_out_dtype, device=q.device)
    elif q_out.shape != shape or not q_out.is_contiguous():
        raise ValueError("q_out: contiguous, of q's shape")
    out_code = _DTYPE_CODE.get(q_out.dtype)
    if out_code is None:
        raise TypeError("q_out is float32 or bfloat16")
    cuda, W = _tables(page_table, seq_lens, tree, B, T)
    if not (cuda and q.is_cuda and k.is_cuda and v.is_cuda and q_out.is_cuda):
        raise _host()
    status = (_lib or lib()).kq_kv_append_tree(
        cache._ref, page_table.data_ptr(), W, seq_lens.data_ptr(), tree.data_ptr(), B, T, q.data_ptr(), k.data_ptr(),
        v.data_ptr(), code, Hq * D if q.is_contiguous() else _row_stride("q", q, B, T, Hq, D),
        heads * D if k.is_contiguous() else _row_stride("k", k, B, T, heads, D),
        heads * D if v.is_contiguous() else _row_stride("v", v, B, T, heads, D), Hq,
        rope._ref, q_out.data_ptr(), out_code, _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_kv_append_tree", status)
    return q_out


def attn_tree_workspace(cache: KVCache, B: int, T: int, n_q_heads: int) -> torch.Tensor:
    """A zero-filled workspace tensor for attn_tree, with room for smaller T and for attn_decode too."""
    n = kq_attn_tree_workspace_size(cache._ref, B, T, n_q_heads)
    if n == 0:
        raise KQError("kq_attn_tree_workspace_size", -4)
    return torch.zeros(n, dtype=torch.uint8, device=cache.k.device)


def attn_tree(cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, tree: torch.Tensor, q: torch.Tensor,
              workspace: torch.Tensor, scale: float | None = None, softcap: float = 0.0, window: int = 0,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """attn_decode of drafted tokens that form a tree (kq_attn_tree), tree [B, T] int64 masks, T up to 64."""
    shape, D, dtype = q.shape, cache.head_dim, q.dtype
    if len(shape) != 4 or shape[3] != D:
        raise ValueError(f"q: [B, T, heads, {D}], not {list(shape)}")
    B, T, Hq, _ = shape
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("q is float32 or bfloat16")
    if out is None:
        out = _new(stream, torch.empty, shape, dtype=dtype, device=q.device)
    elif out.shape != shape or out.dtype is not dtype or not out.is_contiguous():
        raise ValueError("out: contiguous, of q's shape and type")
    cuda, W = _tables(page_table, seq_lens, tree, B, T)
    if workspace.dtype is not _u8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8")
    if not (cuda and q.is_cuda and out.is_cuda and workspace.is_cuda):
        raise _host()
    status = (_lib or lib()).kq_attn_tree(
        cache._ref, page_table.data_ptr(), W, seq_lens.data_ptr(), tree.data_ptr(), B, T, q.data_ptr(), code,
        Hq * D if q.is_contiguous() else _row_stride("q", q, B, T, Hq, D), Hq, D ** -0.5 if scale is None else scale, softcap,
        window, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_attn_tree", status)
    return out


def tree_accept(caches: CacheSet, page_table: torch.Tensor, seq_lens: torch.Tensor, tree: torch.Tensor, tokens: torch.Tensor,
                ids: torch.Tensor, path=None, count=None, next_ids=None, new_lens=None, stream=None):
    """The walk along a verified tree and the accepted branch's slots moved together in all layers' caches (kq_tree_accept,
    kq_latent_accept): tokens [B, T] int32 the nodes' words, ids [B, T] int32 the model's word after each node.  Returns
    (path [B, T], count [B], next_ids [B], new_lens [B]), int32."""
    B, T = shape = tree.shape
    cuda, W = _tables(page_table, seq_lens, tree, B, T)
    if path is None:
        path = _new(stream, torch.empty, (B, T), dtype=_i32, device=tree.device)
    if count is None:
        count = _new(stream, torch.empty, B, dtype=_i32, device=tree.device)
    if next_ids is None:
        next_ids = _new(stream, torch.empty, B, dtype=_i32, device=tree.device)
    if new_lens is None:
        new_lens = _new(stream, torch.empty, B, dtype=_i32, device=tree.device)
    for x, want in ((tokens, shape), (ids, shape), (path, shape), (count, shape[:1]), (next_ids, shape[:1]), (new_lens, shape[:1])):
        if x.dtype is not _i32 or x.shape != want or not x.is_contiguous():
            raise ValueError(f"tokens, ids, path: contiguous int32 [{B}, {T}]; count, next_ids, new_lens: [{B}]")
        cuda = cuda and x.is_cuda
    if not cuda:
        raise _host()
    name = "kq_latent_accept" if caches.latent else "kq_tree_accept"
    status = getattr(_lib or lib(), name)(
        caches._ref, caches.n, page_table.data_ptr(), W, seq_lens.data_ptr(), tree.data_ptr(), tokens.data_ptr(),
        ids.data_ptr(), B, T, path.data_ptr(), count.data_ptr(), next_ids.data_ptr(), new_lens.data_ptr(),
        _here() if stream is None else _stream(stream))
    if status:
        raise KQError(name, status)
    return path, count, next_ids, new_lens


def latent_append(cache: LatentCache, page_table: torch.Tensor, seq_lens: torch.Tensor, q_latent: torch.Tensor,
                  q_rope: torch.Tensor, c: torch.Tensor, rope: RopeNorm, tree: torch.Tensor | None = None,
                  q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kq_latent_append for q_latent [B, T, heads, latent_dim], q_rope [B, T, heads, rope_dim] (a view into the queries'
    product will do) and c [B, T, latent_dim + rope_dim]; rope's k_norm norms the latent.  Returns q_out
    [B, T, heads, latent_dim + rope_dim] bfloat16."""
    shape, C, R, dtype = q_latent.shape, cache.latent_dim, cache.rope_dim, q_latent.dtype
    if len(shape) != 4 or shape[3] != C:
        raise ValueError(f"q_latent: [B, T, heads, {C}], not {list(shape)}")
    B, T, H, _ = shape
    if q_rope.shape != (B, T, H, R) or c.shape != (B, T, C + R) or q_rope.dtype is not dtype or c.dtype is not dtype:
        raise ValueError(f"q_rope: [{B}, {T}, {H}, {R}], c: [{B}, {T}, {C + R}], of q_latent's type")
    code = _DTYPE_CODE.get(dtype)
    if code is None:
        raise TypeError("q_latent, q_rope and c are float32 or bfloat16")
    if rope.q_norm is not None or (rope.norm_dim != 0 and rope.norm_dim != C):
        raise ValueError("norm weights: k_norm [latent_dim]")
    if q_out is None:
        q_out = _new(stream, torch.empty, (B, T, H, C + R), dtype=torch.bfloat16, device=c.device)
    elif q_out.shape != (B, T, H, C + R) or q_out.dtype is not torch.bfloat16 or not q_out.is_contiguous():
        raise ValueError(f"q_out: contiguous bfloat16 [{B}, {T}, {H}, {C + R}]")
    s0, s1, s2, s3 = q_rope.stride()
    if s3 != 1 or (s0 != T * s1 and B > 1 and T > 1):
        raise ValueError("q_rope: tokens at one stride, values contiguous")
    cuda, W = _tables(page_table, seq_lens, tree, B, T)
    if not (cuda and q_latent.is_cuda and q_rope.is_cuda and c.is_cuda and q_out.is_cuda):
        raise _host()
    status = (_lib or lib()).kq_latent_append(
        cache._ref, page_table.data_ptr(), W, seq_lens.data_ptr(), None if tree is None else tree.data_ptr(), B, T,
        q_latent.data_ptr(), q_rope.data_ptr(), c.data_ptr(), code,
        H * C if q_latent.is_contiguous() else _row_stride("q_latent", q_latent, B, T, H, C),
        s1 if T > 1 else s0 if B > 1 else 0, s2 if H > 1 else 0,
        C + R if c.is_contiguous() else _row_stride("c", c.unsqueeze(2), B, T, 1, C + R), H, rope._ref, q_out.data_ptr(),
        _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_latent_append", status)
    return q_out


def latent_attn_workspace(cache: LatentCache, B: int, T: int, n_heads: int) -> torch.Tensor:
    """A zero-filled workspace tensor for latent_attn."""
    n = kq_latent_attn_workspace_size(cache._ref, B, T, n_heads)
    if n == 0:
        raise KQError("kq_latent_attn_workspace_size", -4)
    return torch.zeros(n, dtype=torch.uint8, device=cache.c.device)


def latent_attn(cache: LatentCache, page_table: torch.Tensor, seq_lens: torch.Tensor, q: torch.Tensor,
                workspace: torch.Tensor, scale: float, tree: torch.Tensor | None = None, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """kq_latent_attn for q [B, T, heads, latent_dim + rope_dim] bfloat16; scale: the expanded heads'.  Returns out
    [B, T, heads, latent_dim] bfloat16."""
    shape, C, W = q.shape, cache.latent_dim, cache.latent_dim + cache.rope_dim
    if len(shape) != 4 or shape[3] != W:
        raise ValueError(f"q: [B, T, heads, {W}], not {list(shape)}")
    if q.dtype is not torch.bfloat16:
        raise TypeError("q is bfloat16")
    B, T, H, _ = shape
    if out is None:
        out = _new(stream, torch.empty, (B, T, H, C), dtype=torch.bfloat16, device=q.device)
    elif out.shape != (B, T, H, C) or out.dtype is not torch.bfloat16 or not out.is_contiguous():
        raise ValueError(f"out: contiguous bfloat16 [{B}, {T}, {H}, {C}]")
    cuda, pages = _tables(page_table, seq_lens, tree, B, T)
    if workspace.dtype is not _u8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8")
    if not (cuda and q.is_cuda and out.is_cuda and workspace.is_cuda):
        raise _host()
    status = (_lib or lib()).kq_latent_attn(
        cache._ref, page_table.data_ptr(), pages, seq_lens.data_ptr(), None if tree is None else tree.data_ptr(), B, T,
        q.data_ptr(), H * W if q.is_contiguous() else _row_stride("q", q, B, T, H, W), H, scale, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_latent_attn", status)
    return out


def sample_workspace(M: int, V: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor for sample."""
    n = kq_sample_workspace_size(M, V)
    if n == 0:
        raise KQError("kq_sample_workspace_size", -4)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None, workspace=None,
           ids=None, probs=None, stream=None):
    """kq_sample for logits [M, V] (rows contiguous) and u [M]; temperature, top_p, min_p [M] fp32 and top_k [M] int32,
    or None.  Returns (ids int32 [M], probs fp32 [M])."""
    shape = logits.shape
    M, V = shape
    row = shape[:1]
    code = _DTYPE_CODE.get(logits.dtype)
    if code is None:
        raise TypeError("logits are float32 or bfloat16")
    stride, one = logits.stride()
    if one != 1 and V > 1:
        raise ValueError("logits: each row contiguous")
    if workspace is None:
        workspace = _new(stream, sample_workspace, M, V, logits.device)
    elif workspace.dtype is not _u8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8")
    if ids is None:
        ids = _new(stream, torch.empty, M, dtype=_i32, device=logits.device)
    if probs is None:
        probs = _new(stream, torch.empty, M, dtype=_f32, device=logits.device)
    cuda = logits.is_cuda and workspace.is_cuda
    at = []
    for t, dtype in ((u, _f32), (temperature, _f32), (top_k, _i32), (top_p, _f32), (min_p, _f32), (ids, _i32), (probs, _f32)):
        if t is None:
            at.append(None)
            continue
        if t.dtype is not dtype or t.shape != row or not t.is_contiguous():
            raise ValueError(f"u, temperature, top_p, min_p, probs: contiguous float32 [{M}]; top_k, ids: int32")
        cuda = cuda and t.is_cuda
        at.append(t.data_ptr())
    if not cuda:
        raise _host()
    status = (_lib or lib()).kq_sample(logits.data_ptr(), code, stride, M, V, *at, workspace.data_ptr(), workspace.numel(),
                                       _here() if stream is None else _stream(stream))
    if status:
        raise KQError("kq_sample", status)
    return ids, probs
