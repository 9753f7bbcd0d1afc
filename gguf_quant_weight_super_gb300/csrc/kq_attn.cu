// kq_attn.cu -- attention of the newest T tokens of each sequence over its
// paged cache:
//   s_j = scale * q . k_j, or softcap * tanh(scale * q . k_j / softcap)
//   o   = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   m = max_j s_j
// over the positions j that the token sees (its own and earlier ones, the
// last `window` of them when window > 0); a token that sees none gets 0.
//
// One warp per (sequence, token, head), one key at a time.
#include "kq_cache.h"

namespace kq {
namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__nv_fp8_e4m3 v) { return static_cast<float>(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <class Q, class C, int D>
__global__ void __launch_bounds__(128) attn_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.B) * a.T * a.Hq) return;
  const int h = static_cast<int>(row % a.Hq), hk = h / a.G;
  const int64_t tok = row / a.Hq;
  const int b = static_cast<int>(tok / a.T), t = static_cast<int>(tok % a.T);
  int len = a.seq_lens[b];
  if (len > (a.max_pages << a.page_shift)) {
    if (lane == 0) record_error(a.err, DEV_ERR_PAGE);
    len = static_cast<int>(a.max_pages << a.page_shift);
  }
  const int pos = len - a.T + t;
  const int first = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
  const Q* qp = static_cast<const Q*>(a.q) + tok * a.q_stride + static_cast<int64_t>(h) * D;
  float q[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = to_f(qp[lane + 32 * i]) * a.c.k_scale;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = first; j <= pos; ++j) {
    const int page = a.page_table[b * a.max_pages + (j >> a.page_shift)];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) record_error(a.err, DEV_ERR_PAGE);
      continue;
    }
    const int64_t off = page * a.c.page_stride + (j & (a.c.page_size - 1)) * a.c.slot_stride + hk * a.c.head_stride;
    const C* k = static_cast<const C*>(a.c.k) + off;
    const C* v = static_cast<const C*>(a.c.v) + off;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += q[i] * to_f(k[lane + 32 * i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= a.scale;
    if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
    const float mn = fmaxf(m, s), c = m == mn ? 1.0f : expf(m - mn), p = s == mn ? 1.0f : expf(s - mn);
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * c + p * to_f(v[lane + 32 * i]);
    m = mn;
  }
  const float inv = l > 0.0f ? a.c.v_scale / l : 0.0f;
  Q* op = static_cast<Q*>(a.out) + row * D;
#pragma unroll
  for (int i = 0; i < E; ++i) put(op + lane + 32 * i, l > 0.0f || l != l ? o[i] * (l != l ? l : inv) : 0.0f);
}

template <class Q, class C>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.Hq;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4)), block(128);
  switch (a.c.head_dim) {
    case 64: return launch_pdl(attn_kernel<Q, C, 64>, grid, block, 0, st, a);
    case 128: return launch_pdl(attn_kernel<Q, C, 128>, grid, block, 0, st, a);
    default: return launch_pdl(attn_kernel<Q, C, 256>, grid, block, 0, st, a);
  }
}

}  // namespace

size_t attn_workspace_bytes(int, int, int64_t, int64_t, int) { return 256; }

cudaError_t launch_attn(const AttnArgs& a, int q_bf16, cudaStream_t st) {
  if (a.c.dtype == KQ_BF16)
    return q_bf16 ? launch_d<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_d<float, __nv_bfloat16>(a, st);
  return q_bf16 ? launch_d<__nv_bfloat16, __nv_fp8_e4m3>(a, st) : launch_d<float, __nv_fp8_e4m3>(a, st);
}

}  // namespace kq
