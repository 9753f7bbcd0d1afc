// kq_api.cu -- the extern "C" entry points of libkq (declared in include/kq.h):
// argument checks, kernel choice, launch, and the device error word.
#include <cmath>
#include <cstdio>
#include <initializer_list>
#include <cstring>

#include "../../include/kq.h"
#include "kq_cache.h"
#include "kq_internal.h"

namespace kq {

// The library's device error word (one per device that loads the library).
__device__ int g_device_error = 0;

namespace {
constexpr int kMaxDevices = 64;
int g_sms[kMaxDevices] = {0};
int* g_err_ptr[kMaxDevices] = {nullptr};
thread_local int t_last_cuda_error = 0;

}  // namespace

int current_device_id() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return (dev >= 0 && dev < kMaxDevices) ? dev : 0;
}

int num_sms() {
  const int dev = current_device_id();
  if (!g_sms[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
    g_sms[dev] = n;
  }
  return g_sms[dev];
}

int* device_error_ptr() {
  const int dev = current_device_id();
  if (!g_err_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
    g_err_ptr[dev] = static_cast<int*>(p);
  }
  return g_err_ptr[dev];
}

static kq_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return KQ_OK;
  t_last_cuda_error = static_cast<int>(e);
  return KQ_ERR_CUDA;
}

static bool valid_type(int t) { return t == KQ_Q4_K || t == KQ_Q5_K || t == KQ_Q6_K || t == KQ_IA4; }
static bool kquant_type(int t) { return t == KQ_Q4_K || t == KQ_Q5_K || t == KQ_Q6_K; }  // unpack, chains
static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace kq

using namespace kq;

extern "C" {

size_t kq_block_bytes(int type) { return valid_type(type) ? static_cast<size_t>(block_bytes_of(type)) : 0; }

kq_status kq_ia4_pack(const uint32_t* q, const uint16_t* scales, const uint16_t* biases, int64_t N, int64_t K,
                      void* blocks, kq_stream_t stream) {
  if (N < 0 || K < 0) return KQ_ERR_ARG;
  if (K % 64) return KQ_ERR_SHAPE;
  if (N == 0 || K == 0) return KQ_OK;
  if (!q || !scales || !biases || !blocks) return KQ_ERR_ARG;
  if (!aligned(q, 4) || !aligned(scales, 2) || !aligned(biases, 2) || !aligned(blocks, 16)) return KQ_ERR_ALIGN;
  return cuda_status(launch_ia4_pack(q, scales, biases, N, K, blocks, reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_unpack(int type, const void* blocks, int64_t n_blocks, uint8_t* codes, int8_t* scales, uint8_t* mins,
                    uint16_t* d_bits, uint16_t* dmin_bits, kq_stream_t stream) {
  if (!kquant_type(type)) return KQ_ERR_TYPE;
  if (n_blocks < 0) return KQ_ERR_ARG;
  if (n_blocks == 0) return KQ_OK;
  if (!blocks) return KQ_ERR_ARG;
  if (!aligned(blocks, 16)) return KQ_ERR_ALIGN;
  return cuda_status(launch_unpack(type, blocks, n_blocks, codes, scales, mins, d_bits, dmin_bits,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_dequant(int type, const void* blocks, float* out, int64_t n, kq_stream_t stream) {
  if (!valid_type(type)) return KQ_ERR_TYPE;
  if (n < 0) return KQ_ERR_ARG;
  if (n % 256) return KQ_ERR_SHAPE;
  if (n == 0) return KQ_OK;
  if (!blocks || !out) return KQ_ERR_ARG;
  if (!aligned(blocks, 16) || !aligned(out, 16)) return KQ_ERR_ALIGN;
  return cuda_status(launch_dequant(type, blocks, out, 0, n / 256, reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_dequant_bf16(int type, const void* blocks, uint16_t* out, int64_t n, kq_stream_t stream) {
  if (!valid_type(type)) return KQ_ERR_TYPE;
  if (n < 0) return KQ_ERR_ARG;
  if (n % 256) return KQ_ERR_SHAPE;
  if (n == 0) return KQ_OK;
  if (!blocks || !out) return KQ_ERR_ARG;
  if (!aligned(blocks, 16) || !aligned(out, 16)) return KQ_ERR_ALIGN;
  return cuda_status(launch_dequant(type, blocks, out, 1, n / 256, reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_matvec(int type, const void* W, const void* x, int x_dtype, float* y, int64_t N, int64_t K, int64_t M,
                    kq_stream_t stream) {
  if (!valid_type(type)) return KQ_ERR_TYPE;
  if (x_dtype != KQ_F32 && x_dtype != KQ_BF16) return KQ_ERR_ARG;
  if (N < 0 || K < 0 || M < 0) return KQ_ERR_ARG;
  if (M > 16) return KQ_ERR_UNSUPPORTED;
  if (K % 32 || K > (int64_t(1) << 24)) return KQ_ERR_SHAPE;
  if (N == 0 || M == 0) return KQ_OK;
  if (!y) return KQ_ERR_ARG;
  if (K == 0) return cuda_status(cudaMemsetAsync(y, 0, sizeof(float) * N * M, reinterpret_cast<cudaStream_t>(stream)));
  if (!W || !x) return KQ_ERR_ARG;
  if (!aligned(W, 16) || !aligned(x, 16) || !aligned(y, 4)) return KQ_ERR_ALIGN;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int bf16 = (x_dtype == KQ_BF16);
  cudaError_t e = cudaErrorNotSupported;
  if (M == 1 || (M <= 4 && bf16)) e = launch_matvec1(type, W, x, bf16, y, N, static_cast<int>(K), st, true, M);
  if (e == cudaErrorNotSupported && bf16 && tc_supported(type, N, static_cast<int>(K), static_cast<int>(M)))
    e = launch_tc(type, W, x, y, N, static_cast<int>(K), static_cast<int>(M), st, true);
  if (e == cudaErrorNotSupported)
    e = launch_gemv_batched(type, W, x, bf16, y, N, static_cast<int>(K), static_cast<int>(M), st, true);
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

static_assert(sizeof(ProgPlan) <= sizeof(kq_chain_plan), "plan storage");

static bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

static kq_status check_chain(const kq_op* ops, int n_ops) {
  if (!ops || n_ops <= 0) return KQ_ERR_ARG;
  int last_wait = 0;
  for (int i = 0; i < n_ops; ++i) {
    const kq_op& o = ops[i];
    if (!kquant_type(o.type)) return KQ_ERR_TYPE;
    if (o.x_dtype != KQ_F32 && o.x_dtype != KQ_BF16) return KQ_ERR_ARG;
    if (o.reserved != 0 || o.N <= 0 || o.K <= 0) return KQ_ERR_ARG;
    if (o.K % 32) return KQ_ERR_SHAPE;
    if (o.K > 16384) return KQ_ERR_UNSUPPORTED;
    if (!o.W || !o.x || !o.y) return KQ_ERR_ARG;
    if (!aligned(o.W, 16) || !aligned(o.x, 16) || !aligned(o.y, 4)) return KQ_ERR_ALIGN;
    if (i > 0 && o.wait_previous) last_wait = i;
    // x may not be an output of an op that can still be running
    for (int j = last_wait; j < i; ++j)
      if (overlaps(o.x, o.K * (o.x_dtype == KQ_BF16 ? 2 : 4), ops[j].y, ops[j].N * 4)) return KQ_ERR_ARG;
  }
  for (int i = 0; i < n_ops; ++i) {
    const size_t yb = ops[i].N * 4;
    for (int j = 0; j < n_ops; ++j) {
      const int64_t nbj = (ops[j].K + 255) / 256;
      if (overlaps(ops[i].y, yb, ops[j].W, nbj * ops[j].N * block_bytes_of(ops[j].type))) return KQ_ERR_ARG;
      if (j != i && overlaps(ops[i].y, yb, ops[j].y, ops[j].N * 4)) return KQ_ERR_ARG;
      if (j <= i && overlaps(ops[i].y, yb, ops[j].x, ops[j].K * (ops[j].x_dtype == KQ_BF16 ? 2 : 4)))
        return KQ_ERR_ARG;
    }
  }
  return KQ_OK;
}

static void to_desc(const kq_op* ops, int n_ops, ProgOpDesc* d) {
  for (int i = 0; i < n_ops; ++i) {
    d[i].type = ops[i].type;
    d[i].x_bf16 = ops[i].x_dtype == KQ_BF16;
    d[i].wait_previous = ops[i].wait_previous != 0;
    d[i].W = ops[i].W;
    d[i].x = ops[i].x;
    d[i].y = ops[i].y;
    d[i].N = ops[i].N;
    d[i].K = ops[i].K;
  }
}

size_t kq_chain_workspace_size(const kq_op* ops, int n_ops) {
  if (check_chain(ops, n_ops) != KQ_OK) return 0;
  ProgOpDesc* d = new ProgOpDesc[n_ops];
  to_desc(ops, n_ops, d);
  const size_t b = prog_workspace_size(d, n_ops);
  delete[] d;
  return b;
}

kq_status kq_chain_prepare(const kq_op* ops, int n_ops, void* workspace, size_t workspace_bytes,
                           kq_chain_plan* plan, kq_stream_t stream) {
  const kq_status st = check_chain(ops, n_ops);
  if (st != KQ_OK) return st;
  if (!plan) return KQ_ERR_ARG;
  if (!workspace || !aligned(workspace, 256)) return KQ_ERR_WORKSPACE;
  ProgOpDesc* d = new ProgOpDesc[n_ops];
  to_desc(ops, n_ops, d);
  const size_t need = prog_workspace_size(d, n_ops);
  if (need == 0) { delete[] d; return KQ_ERR_UNSUPPORTED; }
  if (workspace_bytes < need) { delete[] d; return KQ_ERR_WORKSPACE; }
  ProgPlan p = {};
  const cudaError_t e = prog_prepare(d, n_ops, workspace, workspace_bytes, &p,
                                     reinterpret_cast<cudaStream_t>(stream));
  delete[] d;
  if (e != cudaSuccess) return cuda_status(e);
  memset(plan, 0, sizeof(*plan));
  memcpy(plan, &p, sizeof(p));
  return KQ_OK;
}

kq_status kq_chain_run(const kq_chain_plan* plan, void* workspace, kq_stream_t stream) {
  if (!plan || !workspace) return KQ_ERR_ARG;
  ProgPlan p;
  memcpy(&p, plan, sizeof(p));
  if (p.n_ops <= 0) return KQ_ERR_ARG;
  cudaError_t e = prog_run(&p, workspace, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

size_t kq_moe_workspace_size(int64_t N, int64_t M, int32_t top_k, int32_t n_experts) {
  if (N <= 0 || M <= 0 || top_k <= 0 || n_experts <= 0 || M * top_k > 512) return 0;
  return moe_layout(N, M, top_k, n_experts).bytes;
}

kq_status kq_moe_matvec(int type, const void* W_experts, int32_t n_experts, const int32_t* expert_ids,
                        const float* gate_w, const void* x, int x_dtype, int x_per_slot, float* y, int64_t N,
                        int64_t K, int64_t M, int32_t top_k, void* workspace, size_t workspace_bytes,
                        kq_stream_t stream) {
  if (!valid_type(type)) return KQ_ERR_TYPE;
  if (x_dtype != KQ_F32 && x_dtype != KQ_BF16) return KQ_ERR_ARG;
  if (N < 0 || K < 0 || M < 0 || top_k <= 0 || n_experts <= 0) return KQ_ERR_ARG;
  if (K % 32) return KQ_ERR_SHAPE;
  if (N == 0 || M == 0) return KQ_OK;
  if (K == 0 || !moe_supported(type, K, M, top_k, n_experts)) return KQ_ERR_UNSUPPORTED;
  if (!W_experts || !expert_ids || !x || !y) return KQ_ERR_ARG;
  if (!aligned(W_experts, 16) || !aligned(x, 16) || !aligned(y, 4) || !aligned(expert_ids, 4) ||
      (gate_w && !aligned(gate_w, 4)))
    return KQ_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < moe_layout(N, M, top_k, n_experts).bytes)
    return KQ_ERR_WORKSPACE;
  cudaError_t e = launch_moe(type, W_experts, n_experts, expert_ids, gate_w, x, x_dtype == KQ_BF16,
                             x_per_slot ? 1 : 0, y, N, static_cast<int>(K), static_cast<int>(M), top_k, workspace,
                             reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return KQ_ERR_UNSUPPORTED;
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_moe_matvec_noalloc(int type, const void* W_experts, int32_t n_experts, const int32_t* expert_ids,
                                const float* gate_w, const void* x, int x_dtype, int x_per_slot, float* y, int64_t N,
                                int64_t K, int64_t M, int32_t top_k, kq_stream_t stream) {
  if (!valid_type(type)) return KQ_ERR_TYPE;
  if (x_dtype != KQ_F32 && x_dtype != KQ_BF16) return KQ_ERR_ARG;
  if (N < 0 || K < 0 || M < 0 || top_k <= 0 || n_experts <= 0) return KQ_ERR_ARG;
  if (K % 32) return KQ_ERR_SHAPE;
  if (N == 0 || M == 0) return KQ_OK;
  if (K == 0 || !moe_supported(type, K, M, top_k, n_experts)) return KQ_ERR_UNSUPPORTED;
  if (moe_layout(N, M, top_k, n_experts).bytes > moe_static_scratch_bytes()) return KQ_ERR_WORKSPACE;
  if (!W_experts || !expert_ids || !x || !y) return KQ_ERR_ARG;
  if (!aligned(W_experts, 16) || !aligned(x, 16) || !aligned(y, 4) || !aligned(expert_ids, 4) ||
      (gate_w && !aligned(gate_w, 4)))
    return KQ_ERR_ALIGN;
  cudaError_t e = launch_moe_static(type, W_experts, n_experts, expert_ids, gate_w, x, x_dtype == KQ_BF16,
                                    x_per_slot ? 1 : 0, y, N, static_cast<int>(K), static_cast<int>(M), top_k,
                                    reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return KQ_ERR_UNSUPPORTED;
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_moe_route(const float* logits, int64_t M, int32_t n_experts, int32_t top_k, int32_t* expert_ids,
                       float* gate_w, void* workspace, size_t workspace_bytes, kq_stream_t stream) {
  if (M < 0 || n_experts <= 0 || top_k <= 0) return KQ_ERR_ARG;
  if (M == 0) return KQ_OK;
  if (!route_supported(M, n_experts, top_k)) return KQ_ERR_UNSUPPORTED;
  if (!logits || !expert_ids || !gate_w) return KQ_ERR_ARG;
  if (!aligned(logits, 4) || !aligned(expert_ids, 4) || !aligned(gate_w, 4)) return KQ_ERR_ALIGN;
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < route_plan_bytes(M, top_k, n_experts)))
    return KQ_ERR_WORKSPACE;
  cudaError_t e = launch_route(logits, static_cast<int>(M), n_experts, top_k, expert_ids, gate_w, workspace,
                               reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

size_t kq_moe_ffn_workspace_size(int64_t H, int64_t F, int64_t SH, int64_t M, int32_t top_k, int32_t n_experts) {
  if (H <= 0 || F <= 0 || SH < 0 || M <= 0 || top_k <= 0 || n_experts <= 0 || M * top_k > 512) return 0;
  return ffn_layout(H, F, SH, M, top_k, n_experts).bytes;
}

kq_status kq_moe_ffn_offsets(int64_t H, int64_t F, int64_t SH, int64_t M, int32_t top_k, int32_t n_experts,
                             size_t* h_offset, size_t* hs_offset) {
  if (!kq_moe_ffn_workspace_size(H, F, SH, M, top_k, n_experts) || !h_offset || !hs_offset) return KQ_ERR_ARG;
  const FfnLayout L = ffn_layout(H, F, SH, M, top_k, n_experts);
  *h_offset = L.h_off;
  *hs_offset = L.hs_off;
  return KQ_OK;
}

kq_status kq_moe_ffn(const kq_moe_ffn_weights* w, const int32_t* expert_ids, const float* gate_w, const void* x,
                     int x_dtype, float* y, int64_t H, int64_t M, int32_t top_k, void* workspace,
                     size_t workspace_bytes, kq_stream_t stream) {
  if (!w) return KQ_ERR_ARG;
  if (!valid_type(w->type_gate_up) || !valid_type(w->type_down)) return KQ_ERR_TYPE;
  if (x_dtype != KQ_F32 && x_dtype != KQ_BF16) return KQ_ERR_ARG;
  if (w->act != KQ_ACT_SILU && w->act != KQ_ACT_GELU_TANH) return KQ_ERR_ARG;
  if (H < 0 || w->F <= 0 || w->SH < 0 || M < 0 || top_k <= 0 || w->n_experts <= 0) return KQ_ERR_ARG;
  if (H % 32 || w->F % 32 || w->SH % 32) return KQ_ERR_SHAPE;
  if (H == 0 || M == 0) return KQ_OK;
  if (!ffn_supported(w->type_gate_up, w->type_down, H, w->F, w->SH, M, top_k, w->n_experts))
    return KQ_ERR_UNSUPPORTED;
  if (!w->W_gate || !w->W_up || !w->W_down || !expert_ids || !gate_w || !x || !y) return KQ_ERR_ARG;
  if (w->SH > 0 && (!w->Ws_gate || !w->Ws_up || !w->Ws_down)) return KQ_ERR_ARG;
  if (!aligned(w->W_gate, 16) || !aligned(w->W_up, 16) || !aligned(w->W_down, 16) || !aligned(x, 16) ||
      !aligned(y, 4) || !aligned(expert_ids, 4) || !aligned(gate_w, 4))
    return KQ_ERR_ALIGN;
  if (w->SH > 0 && (!aligned(w->Ws_gate, 16) || !aligned(w->Ws_up, 16) || !aligned(w->Ws_down, 16)))
    return KQ_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < ffn_layout(H, w->F, w->SH, M, top_k, w->n_experts).bytes)
    return KQ_ERR_WORKSPACE;
  FfnWeights fw;
  fw.type_gu = w->type_gate_up;
  fw.type_dn = w->type_down;
  fw.n_experts = w->n_experts;
  fw.act = w->act;
  fw.F = w->F;
  fw.SH = w->SH;
  fw.W_gate = w->W_gate;
  fw.W_up = w->W_up;
  fw.W_down = w->W_down;
  fw.Ws_gate = w->Ws_gate;
  fw.Ws_up = w->Ws_up;
  fw.Ws_down = w->Ws_down;
  cudaError_t e = launch_moe_ffn(fw, expert_ids, gate_w, x, x_dtype == KQ_BF16, y, H, static_cast<int>(M), top_k,
                                 workspace, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return KQ_ERR_UNSUPPORTED;
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

static bool cache_dtype(int d) { return d == KQ_BF16 || d == KQ_F8E4M3; }
static bool float_dtype(int d) { return d == KQ_F32 || d == KQ_BF16; }
static bool good_scale(float s) { return s > 0.0f && s <= 3.402823466e38f; }
// a byte stride that is not negative and keeps 16-byte alignment
static bool stride16(int64_t elements, int size) {
  return elements >= 0 && elements < (int64_t(1) << 56) && elements * size % 16 == 0;
}

static kq_status check_cache(const kq_kv_cache* c) {
  if (!c) return KQ_ERR_ARG;
  if (!cache_dtype(c->dtype) || c->n_kv_heads <= 0 || c->n_pages < 0 || c->page_size <= 0) return KQ_ERR_ARG;
  if (!good_scale(c->k_scale) || !good_scale(c->v_scale)) return KQ_ERR_ARG;
  if (c->page_size > 1024 || (c->page_size & (c->page_size - 1)) || !head_dim_supported(c->head_dim) ||
      c->n_kv_heads > 65536 || c->n_pages > INT32_MAX)
    return KQ_ERR_UNSUPPORTED;
  if (c->n_pages > 0 && (!c->k || !c->v)) return KQ_ERR_ARG;
  const int es = c->dtype == KQ_BF16 ? 2 : 1;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !stride16(c->page_stride, es) || !stride16(c->slot_stride, es) ||
      !stride16(c->head_stride, es))
    return KQ_ERR_ALIGN;
  return KQ_OK;
}

static int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

static kq_status kv_append(const kq_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                           const int32_t* seq_lens, const uint64_t* tree, int64_t B, int64_t T, const void* q,
                           const void* k, const void* v, int x_dtype, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, int32_t n_q_heads, const kq_rope* rope, void* q_out, int q_out_dtype,
                           kq_stream_t stream) {
  const kq_status cs = check_cache(cache);
  if (cs != KQ_OK) return cs;
  if (!rope || !float_dtype(x_dtype) || !float_dtype(q_out_dtype)) return KQ_ERR_ARG;
  if (max_pages < 0 || B < 0 || T < 0 || n_q_heads <= 0 || rope->n_positions < 0 || rope->rot_dim < 0) return KQ_ERR_ARG;
  if (rope->rot_dim % 8 || rope->rot_dim > cache->head_dim) return KQ_ERR_SHAPE;
  if (B == 0 || T == 0) return KQ_OK;
  const int64_t heads = int64_t(n_q_heads) + 2 * int64_t(cache->n_kv_heads);
  if (B > INT32_MAX || T > INT32_MAX || B * T > INT32_MAX / heads) return KQ_ERR_UNSUPPORTED;
  if (!seq_lens || !q || !k || !v || !q_out || (max_pages > 0 && !page_table) || (rope->rot_dim > 0 && !rope->cos_sin))
    return KQ_ERR_ARG;
  const int xs = x_dtype == KQ_BF16 ? 2 : 4;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(rope->q_norm, 16) || !aligned(rope->k_norm, 16) ||
      !aligned(rope->cos_sin, 16) || !stride16(q_stride, xs) || !stride16(k_stride, xs) || !stride16(v_stride, xs))
    return KQ_ERR_ALIGN;
  AppendArgs a;
  a.c = *cache;
  a.rope = *rope;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.Hq = n_q_heads;
  a.page_shift = log2_of(cache->page_size);
  a.err = device_error_ptr();
  a.tree = tree;
  cudaError_t e = launch_kv_append(a, x_dtype == KQ_BF16, q_out_dtype == KQ_BF16, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_kv_append(const kq_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                       const int32_t* seq_lens, int64_t B, int64_t T, const void* q, const void* k, const void* v,
                       int x_dtype, int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t n_q_heads,
                       const kq_rope* rope, void* q_out, int q_out_dtype, kq_stream_t stream) {
  return kv_append(cache, page_table, max_pages, seq_lens, nullptr, B, T, q, k, v, x_dtype, q_stride, k_stride, v_stride,
                   n_q_heads, rope, q_out, q_out_dtype, stream);
}

// A tree's masks for T tokens of each of B sequences (either may be 0: nothing to do).
static kq_status check_tree(const uint64_t* tree, int64_t B, int64_t T) {
  if (B < 0 || T < 0) return KQ_ERR_ARG;
  if (T > kMaxTree) return KQ_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return KQ_OK;
  if (!tree) return KQ_ERR_ARG;
  return aligned(tree, 8) ? KQ_OK : KQ_ERR_ALIGN;
}

kq_status kq_kv_append_tree(const kq_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                            const int32_t* seq_lens, const uint64_t* tree, int64_t B, int64_t T, const void* q,
                            const void* k, const void* v, int x_dtype, int64_t q_stride, int64_t k_stride,
                            int64_t v_stride, int32_t n_q_heads, const kq_rope* rope, void* q_out, int q_out_dtype,
                            kq_stream_t stream) {
  const kq_status ts = check_tree(tree, B, T);
  if (ts != KQ_OK) return ts;
  return kv_append(cache, page_table, max_pages, seq_lens, tree, B, T, q, k, v, x_dtype, q_stride, k_stride, v_stride,
                   n_q_heads, rope, q_out, q_out_dtype, stream);
}

static kq_status check_attn(const kq_kv_cache* cache, int64_t B, int64_t T, int32_t n_q_heads, int most = 16) {
  const kq_status cs = check_cache(cache);
  if (cs != KQ_OK) return cs;
  if (B < 0 || T < 0 || n_q_heads <= 0 || n_q_heads % cache->n_kv_heads) return KQ_ERR_ARG;
  if (B > kMaxSeqs || T > most || n_q_heads / cache->n_kv_heads > 16) return KQ_ERR_UNSUPPORTED;
  return KQ_OK;
}

size_t kq_attn_workspace_size(const kq_kv_cache* cache, int64_t B, int64_t T, int32_t n_q_heads) {
  if (check_attn(cache, B, T, n_q_heads) != KQ_OK) return 0;
  return attn_workspace_bytes(cache->head_dim, cache->n_kv_heads, T, n_q_heads);
}

size_t kq_attn_tree_workspace_size(const kq_kv_cache* cache, int64_t B, int64_t T, int32_t n_q_heads) {
  if (check_attn(cache, B, T, n_q_heads, kMaxTree) != KQ_OK) return 0;
  size_t most = 0;  // which kernel takes a call, and how many rows at a time, depends on T: room for any up to it
  for (int64_t t = 0; t <= T; ++t) {
    const size_t n = attn_tree_workspace_bytes(cache->head_dim, cache->n_kv_heads, t, n_q_heads);
    most = n > most ? n : most;
  }
  return most;
}

// most: tokens of a sequence that the call takes.  (An empty batch's tree may be NULL, so tree does not say which call it is.)
static kq_status attn(const kq_kv_cache* cache, const int32_t* page_table, int64_t max_pages, const int32_t* seq_lens,
                      const uint64_t* tree, int most, int64_t B, int64_t T, const void* q, int q_dtype, int64_t q_stride,
                      int32_t n_q_heads, float scale, float softcap, int32_t window, void* out, void* workspace,
                      size_t workspace_bytes, kq_stream_t stream) {
  const kq_status cs = check_attn(cache, B, T, n_q_heads, most);
  if (cs != KQ_OK) return cs;
  if (!float_dtype(q_dtype) || max_pages < 0 || window < 0 || !(softcap == 0.0f || good_scale(softcap)) ||
      !good_scale(scale == 0.0f ? 1.0f : fabsf(scale)))
    return KQ_ERR_ARG;
  if (B == 0 || T == 0) return KQ_OK;
  if (max_pages > INT32_MAX) return KQ_ERR_UNSUPPORTED;
  if (!seq_lens || !q || !out || (max_pages > 0 && !page_table)) return KQ_ERR_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
      !stride16(q_stride, q_dtype == KQ_BF16 ? 2 : 4))
    return KQ_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < (tree ? attn_tree_workspace_bytes : attn_workspace_bytes)(cache->head_dim, cache->n_kv_heads, T, n_q_heads))
    return KQ_ERR_WORKSPACE;
  AttnArgs a;
  a.c = *cache;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.scale = scale;
  a.softcap = softcap;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.Hq = n_q_heads;
  a.G = n_q_heads / cache->n_kv_heads;
  a.page_shift = log2_of(cache->page_size);
  a.room = static_cast<int>(min_i64(max_pages << a.page_shift, kMaxPositions));
  // a window of all positions cuts nothing (of a tree: one of more, as padding stands before them); position - window stays in
  // 32 bits
  a.window = window < a.room + (tree ? 1 : 0) ? window : 0;
  a.ws = workspace;
  a.err = device_error_ptr();
  a.tree = tree;
  cudaError_t e = launch_attn(a, q_dtype == KQ_BF16, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return KQ_ERR_UNSUPPORTED;
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_attn_decode(const kq_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                         const int32_t* seq_lens, int64_t B, int64_t T, const void* q, int q_dtype, int64_t q_stride,
                         int32_t n_q_heads, float scale, float softcap, int32_t window, void* out, void* workspace,
                         size_t workspace_bytes, kq_stream_t stream) {
  return attn(cache, page_table, max_pages, seq_lens, nullptr, 16, B, T, q, q_dtype, q_stride, n_q_heads, scale, softcap,
              window, out, workspace, workspace_bytes, stream);
}

kq_status kq_attn_tree(const kq_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                       const int32_t* seq_lens, const uint64_t* tree, int64_t B, int64_t T, const void* q, int q_dtype,
                       int64_t q_stride, int32_t n_q_heads, float scale, float softcap, int32_t window, void* out,
                       void* workspace, size_t workspace_bytes, kq_stream_t stream) {
  const kq_status ts = check_tree(tree, B, T);
  if (ts != KQ_OK) return ts;
  return attn(cache, page_table, max_pages, seq_lens, tree, kMaxTree, B, T, q, q_dtype, q_stride, n_q_heads, scale, softcap,
              window, out, workspace, workspace_bytes, stream);
}

static kq_status check_latent(const kq_latent_cache* c) {
  if (!c) return KQ_ERR_ARG;
  if (!cache_dtype(c->dtype) || c->n_pages < 0 || c->page_size <= 0 || !good_scale(c->scale)) return KQ_ERR_ARG;
  if (c->page_size > 1024 || (c->page_size & (c->page_size - 1)) || (c->latent_dim != 256 && c->latent_dim != 512) ||
      (c->rope_dim != 32 && c->rope_dim != 64) || c->n_pages > INT32_MAX)
    return KQ_ERR_UNSUPPORTED;
  if (c->n_pages > 0 && !c->c) return KQ_ERR_ARG;
  const int es = c->dtype == KQ_BF16 ? 2 : 1;
  if (!aligned(c->c, 16) || !stride16(c->page_stride, es) || !stride16(c->slot_stride, es)) return KQ_ERR_ALIGN;
  return KQ_OK;
}

// Whether two of n <= kMaxPools addresses (none NULL) are the same, by a table half full at most: 72 of them take 0.2 us of the
// host, 256 take 0.6; compared in pairs 2 and 24.
static bool any_twice(void* const* p, int n) {
  constexpr int ROOM = 2 * kMaxPools;
  const void* seen[ROOM] = {};
  for (int i = 0; i < n; ++i) {
    unsigned at = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p[i]) * 0x9E3779B97F4A7C15ull >> 32) % ROOM;  // (the golden ratio)
    for (; seen[at]; at = (at + 1) % ROOM)
      if (seen[at] == p[i]) return true;
    seen[at] = p[i];
  }
  return false;
}

// The walk; a: the pools' geometry and addresses.
static kq_status accept(TreeArgs& a, const int32_t* page_table, int64_t max_pages, const int32_t* seq_lens,
                        const uint64_t* tree, const int32_t* tokens, const int32_t* ids, int64_t B, int64_t T,
                        int32_t* path, int32_t* count, int32_t* next, int32_t* new_lens, kq_stream_t stream) {
  const kq_status ts = check_tree(tree, B, T);
  if (ts != KQ_OK) return ts;
  if (max_pages < 0) return KQ_ERR_ARG;
  if (B > 65535) return KQ_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return KQ_OK;
  if (!seq_lens || !tokens || !ids || (a.n_pools > 0 && max_pages > 0 && !page_table)) return KQ_ERR_ARG;
  for (const void* p : {static_cast<const void*>(page_table), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(tokens), static_cast<const void*>(ids), static_cast<const void*>(path),
                        static_cast<const void*>(count), static_cast<const void*>(next), static_cast<const void*>(new_lens)})
    if (!aligned(p, 4)) return KQ_ERR_ALIGN;
  // every block walks by itself, whatever another has written; and moves by itself
  for (const int32_t* out : {path, count, next, new_lens})
    if (out && (out == seq_lens || out == tokens || out == ids || out == page_table || static_cast<const void*>(out) == tree))
      return KQ_ERR_ARG;
  if (a.n_pages > 0 && any_twice(a.pool, a.n_pools)) return KQ_ERR_ARG;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.tree = tree;
  a.tokens = tokens;
  a.ids = ids;
  a.path = path;
  a.count = count;
  a.next = next;
  a.new_lens = new_lens;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.err = device_error_ptr();
  cudaError_t e = launch_tree_accept(a, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_tree_accept(const kq_kv_cache* caches, int32_t n_caches, const int32_t* page_table, int64_t max_pages,
                         const int32_t* seq_lens, const uint64_t* tree, const int32_t* tokens, const int32_t* ids,
                         int64_t B, int64_t T, int32_t* path, int32_t* count, int32_t* next, int32_t* new_lens,
                         kq_stream_t stream) {
  if (n_caches < 0 || (n_caches > 0 && !caches)) return KQ_ERR_ARG;
  if (2 * int64_t(n_caches) > kMaxPools) return KQ_ERR_UNSUPPORTED;
  TreeArgs a = {};
  for (int i = 0; i < n_caches; ++i) {
    const kq_kv_cache &c = caches[i], &f = caches[0];
    const kq_status cs = check_cache(&c);
    if (cs != KQ_OK) return cs;
    if (c.dtype != f.dtype || c.n_kv_heads != f.n_kv_heads || c.head_dim != f.head_dim || c.page_size != f.page_size ||
        c.n_pages != f.n_pages || c.page_stride != f.page_stride || c.slot_stride != f.slot_stride ||
        c.head_stride != f.head_stride)
      return KQ_ERR_ARG;
    a.pool[a.n_pools++] = c.k;
    a.pool[a.n_pools++] = c.v;
  }
  if (n_caches > 0) {
    const kq_kv_cache& f = caches[0];
    const int es = f.dtype == KQ_BF16 ? 2 : 1;
    a.n_pages = f.n_pages;
    a.page_stride = f.page_stride * es;
    a.slot_stride = f.slot_stride * es;
    a.head_stride = f.head_stride * es;
    a.head_cols = f.head_dim * es / 16;
    if (int64_t(f.n_kv_heads) * a.head_cols * a.n_pools > INT32_MAX - 4096) return KQ_ERR_UNSUPPORTED;
    a.cols = f.n_kv_heads * a.head_cols;
    a.page_shift = log2_of(f.page_size);
  }
  return accept(a, page_table, max_pages, seq_lens, tree, tokens, ids, B, T, path, count, next, new_lens, stream);
}

kq_status kq_latent_accept(const kq_latent_cache* caches, int32_t n_caches, const int32_t* page_table,
                           int64_t max_pages, const int32_t* seq_lens, const uint64_t* tree, const int32_t* tokens,
                           const int32_t* ids, int64_t B, int64_t T, int32_t* path, int32_t* count, int32_t* next,
                           int32_t* new_lens, kq_stream_t stream) {
  if (n_caches < 0 || (n_caches > 0 && !caches)) return KQ_ERR_ARG;
  if (n_caches > kMaxPools) return KQ_ERR_UNSUPPORTED;
  TreeArgs a = {};
  for (int i = 0; i < n_caches; ++i) {
    const kq_latent_cache &c = caches[i], &f = caches[0];
    const kq_status cs = check_latent(&c);
    if (cs != KQ_OK) return cs;
    if (c.dtype != f.dtype || c.latent_dim != f.latent_dim || c.rope_dim != f.rope_dim || c.page_size != f.page_size ||
        c.n_pages != f.n_pages || c.page_stride != f.page_stride || c.slot_stride != f.slot_stride)
      return KQ_ERR_ARG;
    a.pool[a.n_pools++] = c.c;
  }
  if (n_caches > 0) {
    const kq_latent_cache& f = caches[0];
    const int es = f.dtype == KQ_BF16 ? 2 : 1;
    a.n_pages = f.n_pages;
    a.page_stride = f.page_stride * es;
    a.slot_stride = f.slot_stride * es;
    a.cols = a.head_cols = (f.latent_dim + f.rope_dim) * es / 16;
    a.page_shift = log2_of(f.page_size);
  }
  return accept(a, page_table, max_pages, seq_lens, tree, tokens, ids, B, T, path, count, next, new_lens, stream);
}

kq_status kq_latent_append(const kq_latent_cache* cache, const int32_t* page_table, int64_t max_pages,
                           const int32_t* seq_lens, const uint64_t* tree, int64_t B, int64_t T, const void* q_latent,
                           const void* q_rope, const void* c, int x_dtype, int64_t q_latent_stride,
                           int64_t q_rope_stride, int64_t q_rope_head_stride, int64_t c_stride, int32_t n_heads,
                           const kq_rope* rope, void* q_out, kq_stream_t stream) {
  const kq_status cs = check_latent(cache);
  if (cs != KQ_OK) return cs;
  if (!rope || rope->q_norm || !float_dtype(x_dtype)) return KQ_ERR_ARG;
  if (max_pages < 0 || B < 0 || T < 0 || n_heads <= 0 || rope->n_positions < 0) return KQ_ERR_ARG;
  if (rope->rot_dim != cache->rope_dim) return KQ_ERR_SHAPE;
  if (tree) {
    const kq_status ts = check_tree(tree, B, T);
    if (ts != KQ_OK) return ts;
  }
  if (B == 0 || T == 0) return KQ_OK;
  if (B > INT32_MAX || T > INT32_MAX || B * T > INT32_MAX / (int64_t(n_heads) + 1)) return KQ_ERR_UNSUPPORTED;
  if (!seq_lens || !q_latent || !q_rope || !c || !q_out || (max_pages > 0 && !page_table) || !rope->cos_sin) return KQ_ERR_ARG;
  const int xs = x_dtype == KQ_BF16 ? 2 : 4;
  if (!aligned(q_latent, 16) || !aligned(q_rope, 16) || !aligned(c, 16) || !aligned(q_out, 16) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(rope->k_norm, 16) || !aligned(rope->cos_sin, 16) || !stride16(q_latent_stride, xs) ||
      !stride16(q_rope_stride, xs) || !stride16(q_rope_head_stride, xs) || !stride16(c_stride, xs))
    return KQ_ERR_ALIGN;
  LatentAppendArgs a;
  a.l = *cache;
  a.rope = *rope;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.tree = tree;
  a.q_latent = q_latent;
  a.q_rope = q_rope;
  a.c = c;
  a.q_latent_stride = q_latent_stride;
  a.q_rope_stride = q_rope_stride;
  a.q_rope_head_stride = q_rope_head_stride;
  a.c_stride = c_stride;
  a.q_out = q_out;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.H = n_heads;
  a.page_shift = log2_of(cache->page_size);
  a.err = device_error_ptr();
  cudaError_t e = launch_latent_append(a, x_dtype == KQ_BF16, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

static kq_status check_latent_attn(const kq_latent_cache* cache, int64_t B, int64_t T, int32_t n_heads) {
  const kq_status cs = check_latent(cache);
  if (cs != KQ_OK) return cs;
  if (B < 0 || T < 0 || n_heads <= 0) return KQ_ERR_ARG;
  return B > kMaxSeqs || T > kMaxTree || n_heads > 256 ? KQ_ERR_UNSUPPORTED : KQ_OK;
}

size_t kq_latent_attn_workspace_size(const kq_latent_cache* cache, int64_t B, int64_t T, int32_t n_heads) {
  if (check_latent_attn(cache, B, T, n_heads) != KQ_OK) return 0;
  return latent_workspace_bytes(*cache, T, n_heads);
}

kq_status kq_latent_attn(const kq_latent_cache* cache, const int32_t* page_table, int64_t max_pages,
                         const int32_t* seq_lens, const uint64_t* tree, int64_t B, int64_t T, const void* q,
                         int64_t q_stride, int32_t n_heads, float scale, void* out, void* workspace,
                         size_t workspace_bytes, kq_stream_t stream) {
  const kq_status cs = check_latent_attn(cache, B, T, n_heads);
  if (cs != KQ_OK) return cs;
  if (max_pages < 0 || !good_scale(scale == 0.0f ? 1.0f : fabsf(scale))) return KQ_ERR_ARG;
  if (B == 0 || T == 0) return KQ_OK;
  if (max_pages > INT32_MAX) return KQ_ERR_UNSUPPORTED;
  const int64_t tiles = (max_pages * cache->page_size + 31) / 32 + 24;  // the line of tiles is counted in 31 bits
  if (tiles * B > INT32_MAX / ((T * n_heads + 63) / 64)) return KQ_ERR_UNSUPPORTED;
  if (!seq_lens || !q || !out || (max_pages > 0 && !page_table)) return KQ_ERR_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(tree, 8) ||
      !stride16(q_stride, 2))
    return KQ_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < latent_workspace_bytes(*cache, T, n_heads))
    return KQ_ERR_WORKSPACE;
  LatentArgs a;
  a.l = *cache;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.tree = tree;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.scale = scale;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.H = n_heads;
  a.page_shift = log2_of(cache->page_size);
  a.room = static_cast<int>(min_i64(max_pages << a.page_shift, kMaxPositions));
  a.ws = workspace;
  a.err = device_error_ptr();
  cudaError_t e = launch_latent(a, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return KQ_ERR_UNSUPPORTED;
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_selftest_attn_ctas(const kq_kv_cache* cache, int64_t B, int64_t T, int q_dtype, int32_t n_q_heads,
                                int* planned, int* resident) {
  const kq_status cs = check_attn(cache, B, T, n_q_heads);
  if (cs != KQ_OK) return cs;
  if (!float_dtype(q_dtype) || B == 0 || T == 0 || !planned || !resident) return KQ_ERR_ARG;
  AttnArgs a = {};
  a.c = *cache;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.Hq = n_q_heads;
  a.G = n_q_heads / cache->n_kv_heads;
  AttnShape s = {0, 0};
  const cudaError_t e = launch_attn(a, q_dtype == KQ_BF16, nullptr, &s);
  *planned = s.planned;
  *resident = s.resident;
  return e == cudaErrorNotSupported ? KQ_ERR_UNSUPPORTED : cuda_status(e);
}

size_t kq_sample_workspace_size(int64_t M, int64_t V) {
  if (M < 0 || V < 1 || M > (1 << 24) || V > (1 << 20)) return 0;
  return sample_workspace_bytes(M, V);
}

kq_status kq_sample(const void* logits, int dtype, int64_t row_stride, int64_t M, int64_t V, const float* u,
                    const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                    int32_t* ids, float* probs, void* workspace, size_t workspace_bytes, kq_stream_t stream) {
  if (!float_dtype(dtype) || M < 0 || V < 0 || row_stride < 0) return KQ_ERR_ARG;
  if (V < 1 || V > (1 << 20) || M > (1 << 24)) return KQ_ERR_UNSUPPORTED;
  if (M == 0) return KQ_OK;
  if (!logits || !u || !ids) return KQ_ERR_ARG;
  if (!aligned(logits, dtype == KQ_BF16 ? 2 : 4) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(ids, 4) || !aligned(probs, 4))
    return KQ_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < sample_workspace_bytes(M, V)) return KQ_ERR_WORKSPACE;
  SampleArgs a;
  a.logits = logits;
  a.row_stride = row_stride;
  a.temperature = temperature;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.top_k = top_k;
  a.ids = ids;
  a.probs = probs;
  a.ws = workspace;
  a.M = static_cast<int>(M);
  a.V = static_cast<int>(V);
  cudaError_t e = launch_sample(a, dtype == KQ_BF16, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaGetLastError();
  return cuda_status(e);
}

kq_status kq_selftest_wait(int kind, int* observed_code, kq_stream_t stream) {
  if ((kind != 0 && kind != 1) || !observed_code) return KQ_ERR_ARG;
  return cuda_status(run_selftest_wait(kind, observed_code, reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_moe_check(void* workspace, kq_stream_t stream) {
  if (!workspace) return KQ_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_status(e);
  if (v) {
    e = cudaMemsetAsync(workspace, 0, sizeof(int), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e);
    return KQ_ERR_DEVICE;
  }
  return KQ_OK;
}

kq_status kq_device_error(int* code, int clear) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int));
  if (e != cudaSuccess) return cuda_status(e);
  if (clear && v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (code) *code = v;
  return v ? KQ_ERR_DEVICE : KQ_OK;
}

int kq_last_cuda_error(void) { return t_last_cuda_error; }

const char* kq_status_string(kq_status s) {
  switch (s) {
    case KQ_OK: return "ok";
    case KQ_ERR_ARG: return "invalid argument";
    case KQ_ERR_TYPE: return "unknown block type";
    case KQ_ERR_SHAPE: return "unsupported shape (K must be a multiple of 32; dequant n a multiple of 256)";
    case KQ_ERR_UNSUPPORTED: return "size outside this call's limits (products: M 1..16, top_k 1..32)";
    case KQ_ERR_ALIGN: return "misaligned pointer";
    case KQ_ERR_CUDA: return "CUDA error";
    case KQ_ERR_WORKSPACE: return "workspace missing or too small";
    case KQ_ERR_DEVICE: return "device error word set";
    default: return "unknown status";
  }
}

}  // extern "C"
