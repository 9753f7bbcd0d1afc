// kq_latent.cu -- attention of the newest T tokens of each sequence over its
// cache of latent vectors c_j, which all heads share, in absorbed form:
//   s_j = scale q.c_j (latent and rope part),  out = sum_j softmax(s)_j c_j[0 .. C)
// A CTA takes one token and HEADS of its heads, and goes over the positions in
// tiles of 32 with a running maximum and running sums, everything in fp32.
#include "kq_cache.h"

namespace kq {
namespace {

constexpr int STH = 256, HEADS = 8, KT = 32;

__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float value(const __nv_fp8_e4m3* p) { return static_cast<float>(*p); }

template <class Y>
__global__ void __launch_bounds__(STH) latent_kernel(const __grid_constant__ LatentArgs a) {
  extern __shared__ float smem[];
  const int C = a.l.latent_dim, W = C + a.l.rope_dim;
  float* tile = smem;               // [KT][W + 1]
  float* q = tile + KT * (W + 1);   // [HEADS][W]
  __shared__ float s[HEADS][KT];    // scores, then weights
  __shared__ float m[HEADS], l[HEADS], fix[HEADS];
  __shared__ int seen[KT];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  const int groups = (a.H + HEADS - 1) / HEADS;
  const int tok = blockIdx.x / groups, h0 = (blockIdx.x - tok * groups) * HEADS, b = tok / a.T, t = tok - b * a.T;
  int len = max(__ldg(a.seq_lens + b), 0);
  if (len > a.room) {
    if (tid == 0) record_error(a.err, DEV_ERR_PAGE);
    len = a.room;
  }
  const int base = len - a.T;
  uint64_t bits = 0;
  int pos = base + t;
  if (a.tree) {
    bits = tree_bits(__ldg(a.tree + tok), a.T, t, len);
    pos = tree_position(bits, a.T, len);
  }
  for (int x = tid; x < HEADS * W; x += STH) {
    const int h = h0 + x / W;
    q[x] = h < a.H ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[tok * a.q_stride + static_cast<int64_t>(h) * W + x % W]) : 0.0f;
  }
  if (tid < HEADS) {
    m[tid] = -INFINITY;
    l[tid] = 0.0f;
  }
  float o[HEADS][2] = {};
  for (int j0 = 0; j0 < len && pos >= 0; j0 += KT) {
    __syncthreads();
    if (tid < KT) {
      const int j = j0 + tid, u = j - base;
      bool see = j < len && (a.tree && u >= 0 ? u < 64 && (bits >> u & 1) : j <= pos);
      if (see) {
        const int page = __ldg(a.page_table + b * a.max_pages + (j >> a.page_shift));
        if (page < 0 || page >= a.l.n_pages) {
          record_error(a.err, DEV_ERR_PAGE);
          see = false;
        }
      }
      seen[tid] = see;
    }
    __syncthreads();
    for (int x = tid; x < KT * W; x += STH) {
      const int k = x / W, d = x - k * W, j = j0 + k;
      float v = 0.0f;
      if (seen[k]) {
        const int page = __ldg(a.page_table + b * a.max_pages + (j >> a.page_shift));
        v = value(static_cast<const Y*>(a.l.c) + page * a.l.page_stride + (j & (a.l.page_size - 1)) * a.l.slot_stride + d) * a.l.scale;
      }
      tile[k * (W + 1) + d] = v;
    }
    __syncthreads();
    for (int x = warp; x < HEADS; x += STH / 32) {  // a lane per position
      float acc = 0.0f;
      for (int d = 0; d < W; ++d) acc = fmaf(q[x * W + d], tile[lane * (W + 1) + d], acc);
      acc = seen[lane] ? acc * a.scale * 1.4426950408889634f : -INFINITY;
      float top = acc;
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
      const float mm = fmaxf(m[x], top), ref = mm == -INFINITY ? 0.0f : mm;
      const float w = exp2f(acc - ref);
      float sum = w;
      for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
      s[x][lane] = w;
      __syncwarp();
      if (lane == 0) {
        fix[x] = exp2f(m[x] - ref);
        l[x] = l[x] * fix[x] + sum;
        m[x] = mm;
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      o[h][0] *= fix[h];
      o[h][1] *= fix[h];
    }
    for (int k = 0; k < KT; ++k) {
      if (!seen[k]) continue;
      for (int i = 0; i < C / STH; ++i) {
        const float v = tile[k * (W + 1) + tid + i * STH];
#pragma unroll
        for (int h = 0; h < HEADS; ++h) o[h][i] = fmaf(s[h][k], v, o[h][i]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < a.H)
      for (int i = 0; i < C / STH; ++i)
        static_cast<__nv_bfloat16*>(a.out)[(static_cast<int64_t>(tok) * a.H + h0 + h) * C + tid + i * STH] =
            __float2bfloat16_rn(l[h] == 0.0f ? 0.0f : o[h][i] / l[h]);
}

template <class Y>
cudaError_t launch_y(const LatentArgs& a, cudaStream_t st) {
  const int W = a.l.latent_dim + a.l.rope_dim, smem = (KT * (W + 1) + HEADS * W) * 4;
  const cudaError_t e = cudaFuncSetAttribute(latent_kernel<Y>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_kernel<Y>, dim3(a.B * a.T * ((a.H + HEADS - 1) / HEADS)), dim3(STH), smem, st, a);
}

}  // namespace

size_t latent_workspace_bytes(const kq_latent_cache&, int64_t, int) { return 256; }

cudaError_t launch_latent(const LatentArgs& a, cudaStream_t st) {
  return a.l.dtype == KQ_BF16 ? launch_y<__nv_bfloat16>(a, st) : launch_y<__nv_fp8_e4m3>(a, st);
}

}  // namespace kq
