// kq_latent_append.cu -- what stands between a latent layer's products and its
// attention, in one launch: the RMS norm of each new token's latent vector, the
// rotation of its rope key and of the queries' rope parts, the vector into the
// sequence's cache page and the queries, latent and rope part side by side, out.
//
//   latent   x / sqrt(mean(x^2) + eps) * (w + off)       (w optional)
//   rope     (a, b) -> (a c - b s, b c + a s), c, s from the table of the position
//
// Everything is fp32 up to one rounding, as in kq_append.cu.  Bound: memory; the
// queries' rows are nearly all of it (each is read once and written once as bf16).
// A warp takes a row, eight neighbouring values of its latent part per lane and
// turn; the R / 8 first lanes the rope part, two vectors of four that are each
// other's rotation partners.
#include "kq_cache.h"
#include "kq_vec.cuh"

namespace kq {
namespace {

constexpr int LTH = 128;  // threads per CTA

struct F8 {
  float4 a, b;
};
__device__ __forceinline__ F8 load8(const float* p) { return {load4(p), load4(p + 4)}; }
__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  return {bf16x4(make_uint2(u.x, u.y)), bf16x4(make_uint2(u.z, u.w))};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, F8 v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v.a.x, v.a.y), bf16_pair(v.a.z, v.a.w), bf16_pair(v.b.x, v.b.y),
                                            bf16_pair(v.b.z, v.b.w));
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, F8 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(v.a), e4m3x4(v.b));
}

// A row's values: the latent part's N vectors of this lane, and the rope part's (lanes below R / 8).
template <int N>
struct Row {
  F8 v[N], r;
};

// X: the inputs; Y: the cache; C, R: latent and rope values; U rows per warp.
template <class X, class Y, int C, int R, int U>
__global__ void __launch_bounds__(LTH) latent_append_kernel(const __grid_constant__ LatentAppendArgs a) {
  constexpr int N = C / 256, W = C + R;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int per = (a.H + 1 + U - 1) / U;  // warps per token; rows: the cache's, then the heads'
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (LTH / 32) + threadIdx.x / 32;
  const int64_t tok = unit / per;
  if (tok >= static_cast<int64_t>(a.B) * a.T) return;
  const int row0 = static_cast<int>(unit - tok * per) * U;
  const int b = static_cast<int>(tok / a.T), t = static_cast<int>(tok - static_cast<int64_t>(b) * a.T);
  const bool turns = lane < R / 8;
  const int e0 = a.rope.interleaved ? 8 * lane : 4 * lane, e1 = a.rope.interleaved ? e0 + 4 : R / 2 + e0;
  Row<N> x[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = row0 + i - 1;
    if (h >= a.H) continue;
    const X* src = h < 0 ? static_cast<const X*>(a.c) + tok * a.c_stride
                         : static_cast<const X*>(a.q_latent) + tok * a.q_latent_stride + static_cast<int64_t>(h) * C;
    const X* rope = h < 0 ? src + C : static_cast<const X*>(a.q_rope) + tok * a.q_rope_stride + h * a.q_rope_head_stride;
#pragma unroll
    for (int n = 0; n < N; ++n) x[i].v[n] = load8(src + 8 * (lane + 32 * n));
    if (turns) x[i].r = {load4(rope + e0), load4(rope + e1)};
  }
  const int len = max(__ldg(a.seq_lens + b), 0), slot = len - a.T + t;
  int pos = slot;  // below 0: padding
  if (a.tree) pos = tree_position(tree_bits(__ldg(a.tree + tok), a.T, t, len), a.T, len);
  bool ok = pos >= 0;
  if (ok && pos >= a.rope.n_positions) {
    if (lane == 0) record_error(a.err, DEV_ERR_POSITION);
    ok = false;
  }
  if (ok && turns) {
    const float* cs = a.rope.cos_sin + static_cast<int64_t>(pos) * R + 4 * lane;
    const float4 c = load4(cs), s = load4(cs + R / 2);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (row0 + i <= a.H) rotate8(x[i].r.a, x[i].r.b, c, s, a.rope.interleaved);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = row0 + i - 1;
    if (h >= a.H) continue;
    if (h >= 0) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.q_out) + (tok * a.H + h) * W;
      const float4 zero = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < N; ++n) store8(dst + 8 * (lane + 32 * n), ok ? x[i].v[n] : F8{zero, zero});
      if (turns) {
        store4(dst + C + e0, ok ? x[i].r.a : zero);
        store4(dst + C + e1, ok ? x[i].r.b : zero);
      }
    } else if (ok) {
      const int64_t pi = slot >> a.page_shift;
      const int page = pi < a.max_pages ? __ldg(a.page_table + b * a.max_pages + pi) : -1;
      if (page < 0 || page >= a.l.n_pages) {
        if (lane == 0) record_error(a.err, DEV_ERR_PAGE);
        continue;
      }
      Y* dst = static_cast<Y*>(a.l.c) + page * a.l.page_stride + (slot & (a.l.page_size - 1)) * a.l.slot_stride;
      if (a.rope.k_norm) {
        float ss = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) ss += sq4(x[i].v[n].a) + sq4(x[i].v[n].b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float f = rsqrtf(ss * (1.0f / C) + a.rope.eps);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const float* w = a.rope.k_norm + 8 * (lane + 32 * n);
          x[i].v[n].a = scale4(x[i].v[n].a, f, load4(w), a.rope.norm_offset);
          x[i].v[n].b = scale4(x[i].v[n].b, f, load4(w + 4), a.rope.norm_offset);
        }
      }
      const float sc = a.l.scale;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (sc != 1.0f) x[i].v[n] = {over4(x[i].v[n].a, sc), over4(x[i].v[n].b, sc)};
        store8(dst + 8 * (lane + 32 * n), x[i].v[n]);
      }
      if (turns) {
        if (sc != 1.0f) x[i].r = {over4(x[i].r.a, sc), over4(x[i].r.b, sc)};
        store4(dst + C + e0, x[i].r.a);
        store4(dst + C + e1, x[i].r.b);
      }
    }
  }
}

template <class X, class Y, int C, int R>
cudaError_t launch_r(const LatentAppendArgs& a, cudaStream_t st) {
  constexpr int U = 1;
  const int64_t warps = static_cast<int64_t>(a.B) * a.T * ((a.H + 1 + U - 1) / U), grid = (warps + LTH / 32 - 1) / (LTH / 32);
  return launch_pdl(latent_append_kernel<X, Y, C, R, U>, dim3(static_cast<unsigned>(grid)), dim3(LTH), 0, st, a);
}
template <class X, class Y>
cudaError_t launch_c(const LatentAppendArgs& a, cudaStream_t st) {
  if (a.l.latent_dim == 512) return a.l.rope_dim == 64 ? launch_r<X, Y, 512, 64>(a, st) : launch_r<X, Y, 512, 32>(a, st);
  return a.l.rope_dim == 64 ? launch_r<X, Y, 256, 64>(a, st) : launch_r<X, Y, 256, 32>(a, st);
}
template <class X>
cudaError_t launch_y(const LatentAppendArgs& a, cudaStream_t st) {
  return a.l.dtype == KQ_BF16 ? launch_c<X, __nv_bfloat16>(a, st) : launch_c<X, __nv_fp8_e4m3>(a, st);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, int x_bf16, cudaStream_t st) {
  return x_bf16 ? launch_y<__nv_bfloat16>(a, st) : launch_y<float>(a, st);
}

}  // namespace kq
