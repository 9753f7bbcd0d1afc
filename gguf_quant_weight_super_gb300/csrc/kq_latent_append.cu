// kq_latent_append.cu -- what stands between a latent layer's products and its
// attention, in one launch: the RMS norm of each new token's latent vector, the
// rotation of its rope key and of the queries' rope parts, the vector into the
// sequence's cache page and the queries, latent and rope part side by side, out.
//
//   latent   x / sqrt(mean(x^2) + eps) * (w + off)       (w optional)
//   rope     (a, b) -> (a c - b s, b c + a s), c, s from the table of the position
//
// Everything is fp32 up to one rounding, as in kq_append.cu.  Bound: memory, and
// nearly the instructions; the queries' rows are nearly all of it (each is read
// once and written once as bf16, without a conversion where it is bf16).  A warp
// takes U rows of a token's queries: of their latent parts eight neighbouring
// values per lane and turn, of their rope parts, side by side in its lanes, two
// vectors of four that are each other's rotation partners.  The cache's row has a
// warp of its own.  Measured on one GB300, calls in a graph: 4 x 2047 tokens of 16
// heads of 512 + 64 values, bf16 into e4m3, 49 us (95% of the copy rate; a warp per row, with
// conversions: 63); one token 2.9 us.
#include "kq_cache.h"
#include "kq_vec.cuh"

namespace kq {
namespace {

constexpr int LTH = 128;  // threads per CTA
constexpr int ROWS = 4;   // of the queries, per warp

// 16 bytes of output: eight bf16 values.
__device__ __forceinline__ uint4 bf16x8(F8 v) {
  return make_uint4(bf16_pair(v.a.x, v.a.y), bf16_pair(v.a.z, v.a.w), bf16_pair(v.b.x, v.b.y), bf16_pair(v.b.z, v.b.w));
}
__device__ __forceinline__ uint4 as_bf16(const float* p) { return bf16x8(load8(p)); }
__device__ __forceinline__ uint4 as_bf16(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// X: the inputs; Y: the cache; C, R: latent and rope values; U rows per warp.
template <class X, class Y, int C, int R, int U>
__global__ void __launch_bounds__(LTH) latent_append_kernel(const __grid_constant__ LatentAppendArgs a) {
  constexpr int N = C / 256, W = C + R, RL = R / 8;  // vectors of a row per lane; lanes of a rope part
  static_assert(U * RL <= 32, "all rope parts at once");
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t per = 1 + (a.H + U - 1) / U;  // warps per token
  const uint32_t unit = blockIdx.x * (LTH / 32) + threadIdx.x / 32, tok = unit / per;
  if (tok >= static_cast<uint32_t>(a.B) * a.T) return;
  const int h0 = (static_cast<int>(unit - tok * per) - 1) * U;  // below 0: the cache's row
  const uint32_t b = tok / a.T, t = tok - b * a.T;
  // the rope part: row h0 + lane / RL (the cache's: lanes below RL)
  const int hr = h0 < 0 ? -1 : h0 + lane / RL, i0 = lane % RL;
  const bool turns = h0 < 0 ? lane < RL : lane < U * RL && hr < a.H;
  const int e0 = a.rope.interleaved ? 8 * i0 : 4 * i0, e1 = a.rope.interleaved ? e0 + 4 : R / 2 + e0;
  const X* crow = static_cast<const X*>(a.c) + static_cast<int64_t>(tok) * a.c_stride;
  F8 r;
  if (turns) {
    const X* src = h0 < 0 ? crow + C : static_cast<const X*>(a.q_rope) + static_cast<int64_t>(tok) * a.q_rope_stride + hr * a.q_rope_head_stride;
    r = {load4(src + e0), load4(src + e1)};
  }
  const int len = max(__ldg(a.seq_lens + b), 0), slot = len - a.T + static_cast<int>(t);
  int pos = slot;  // below 0: padding
  if (a.tree) pos = tree_position(tree_bits(__ldg(a.tree + tok), a.T, t, len), a.T, len);
  bool ok = pos >= 0;
  if (ok && pos >= a.rope.n_positions) {
    if (lane == 0) record_error(a.err, DEV_ERR_POSITION);
    ok = false;
  }
  if (ok && turns) {
    const float* cs = a.rope.cos_sin + static_cast<int64_t>(pos) * R + 4 * i0;
    rotate8(r.a, r.b, load4(cs), load4(cs + R / 2), a.rope.interleaved);
  }
  if (h0 >= 0) {
    constexpr int FLY = U < 2 || sizeof(X) == 2 ? U : 2;  // rows in flight
    const X* src = static_cast<const X*>(a.q_latent) + static_cast<int64_t>(tok) * a.q_latent_stride + static_cast<int64_t>(h0) * C + 8 * lane;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.q_out) + (static_cast<int64_t>(tok) * a.H + h0) * W;
#pragma unroll
    for (int u0 = 0; u0 < U; u0 += FLY) {
      uint4 x[FLY][N];
#pragma unroll
      for (int u = 0; u < FLY; ++u)
#pragma unroll
        for (int n = 0; n < N; ++n)
          x[u][n] = ok && h0 + u0 + u < a.H ? as_bf16(src + (u0 + u) * C + 256 * n) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < FLY; ++u)
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (h0 + u0 + u < a.H) *reinterpret_cast<uint4*>(dst + (u0 + u) * W + 8 * lane + 256 * n) = x[u][n];
    }
    if (turns) {
      const float4 zero = make_float4(0, 0, 0, 0);
      dst += (lane / RL) * W + C;
      store4(dst + e0, ok ? r.a : zero);
      store4(dst + e1, ok ? r.b : zero);
    }
    return;
  }
  if (!ok) return;
  const int64_t pi = slot >> a.page_shift;
  const int page = pi < a.max_pages ? __ldg(a.page_table + b * a.max_pages + pi) : -1;
  if (page < 0 || page >= a.l.n_pages) {
    if (lane == 0) record_error(a.err, DEV_ERR_PAGE);
    return;
  }
  F8 v[N];
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = load8(crow + 8 * (lane + 32 * n));
  Y* dst = static_cast<Y*>(a.l.c) + page * a.l.page_stride + (slot & (a.l.page_size - 1)) * a.l.slot_stride;
  if (a.rope.k_norm) {
    float ss = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) ss += sq4(v[n].a) + sq4(v[n].b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float f = rsqrtf(ss * (1.0f / C) + a.rope.eps);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const F8 w = load8(a.rope.k_norm + 8 * (lane + 32 * n));
      v[n] = {scale4(v[n].a, f, w.a, a.rope.norm_offset), scale4(v[n].b, f, w.b, a.rope.norm_offset)};
    }
  }
  const float sc = a.l.scale;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (sc != 1.0f) v[n] = {over4(v[n].a, sc), over4(v[n].b, sc)};
    store8(dst + 8 * (lane + 32 * n), v[n]);
  }
  if (turns) {
    if (sc != 1.0f) r = {over4(r.a, sc), over4(r.b, sc)};
    store4(dst + C + e0, r.a);
    store4(dst + C + e1, r.b);
  }
}

template <class X, class Y, int C, int R, int U>
cudaError_t launch_u(const LatentAppendArgs& a, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(a.B) * a.T * (1 + (a.H + U - 1) / U), grid = (warps + LTH / 32 - 1) / (LTH / 32);
  return launch_pdl(latent_append_kernel<X, Y, C, R, U>, dim3(static_cast<unsigned>(grid)), dim3(LTH), 0, st, a);
}
template <class X, class Y, int C, int R>
cudaError_t launch_r(const LatentAppendArgs& a, cudaStream_t st) {
  // several rows per warp once that still fills the device (8 CTAs per SM)
  const int64_t few = static_cast<int64_t>(a.B) * a.T * (1 + (a.H + ROWS - 1) / ROWS) / (LTH / 32);
  return few >= 8 * num_sms() ? launch_u<X, Y, C, R, ROWS>(a, st) : launch_u<X, Y, C, R, 1>(a, st);
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
