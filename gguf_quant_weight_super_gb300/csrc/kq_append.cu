// kq_append.cu -- what stands between a layer's q|k|v products and its
// attention, in one launch: RMS norms of q and k per head, the rotation by
// position, q out, and k and v into the sequences' cache pages.
//
//   y = x / sqrt(mean(x^2) + eps) * (w + off)             (q and k, optional)
//   (a, b) -> (a c - b s, b c + a s)                      (q and k, first rot_dim values)
//
// with c, s read from a table of cos | sin per position: the angles of long
// contexts (positions of 10^5 and more, scaled frequencies) lose their digits
// in fp32 products, so they are made once, by the caller, in 64 bits.
//
// Everything is fp32 up to one rounding into q_out or the cache; an 8-bit
// cache stores x / scale, saturated at e4m3's largest value 448 (a NaN stays
// a NaN).
//
// Bound: memory (and at one token, the chain of dependent loads length ->
// page id -> store).  A row of D values is D / 8 lanes' work: each lane holds
// two vectors of four values that are each other's rotation partners (i and
// i + rot/2, or adjacent pairs when interleaved), so the rotation needs no
// exchange between lanes and the norm one shuffle sum over the row's lanes.
// Each group of lanes takes three heads of a token, whose loads are all in
// flight together, and reads the token's cosines and sines once for them.  With
// few tokens a group takes one head, so that the rows spread over more SMs.
// Measured on one GB300, calls in a graph: 4 x 2047 tokens of 24 heads of 256,
// fp32 into e4m3, 50 us (5.8 TB/s, 86% of the copy rate; with two heads per
// group 53, with six 58, with 256 threads 55; a CTA per token 48, but then 28917
// tokens of 6 heads, bf16, 46 in place of 28); one token of 48 heads 2.1 us.
#include "kq_cache.h"

namespace kq {
namespace {

constexpr int ATH = 128;  // threads per CTA
constexpr int ROWS = 3;   // rows per group of lanes at a time

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
}
__device__ __forceinline__ void store4(__nv_fp8_e4m3* p, float4 v) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z, v.w), __NV_SATFINITE, __NV_E4M3);
  *reinterpret_cast<uint32_t*>(p) = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ float sq4(float4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }
__device__ __forceinline__ float4 scale4(float4 v, float s, float4 w, float off) {
  return make_float4(v.x * s * (w.x + off), v.y * s * (w.y + off), v.z * s * (w.z + off), v.w * s * (w.w + off));
}

// X: q, k, v; O: q_out; C: the cache.  LG = D / 8 lanes hold one row; U rows per group of lanes.
template <class X, class O, class C, int LG, int U>
__global__ void __launch_bounds__(ATH) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int D = 8 * LG, NG = ATH / LG;
  pdl_wait();
  pdl_launch_dependents();
  const int Hkv = a.c.n_kv_heads, H = a.Hq + 2 * Hkv;
  const uint32_t per = (H + U - 1) / U;  // groups per token
  const uint32_t grp = blockIdx.x * NG + threadIdx.x / LG, all = static_cast<uint32_t>(a.B) * a.T * per;
  const uint32_t tok = min(grp, all - 1) / per;  // groups past the last: its token, no head
  const int h0 = grp < all ? static_cast<int>(grp - tok * per) * U : H;
  const int b = tok / a.T, t = tok - b * a.T;
  const int l = threadIdx.x % LG;
  const int rot = a.rope.rot_dim, rl = rot / 8;
  // the row's two vectors of this lane
  int e0, e1;
  if (l >= rl || a.rope.interleaved) {
    e0 = 8 * l;
    e1 = e0 + 4;
  } else {
    e0 = 4 * l;
    e1 = rot / 2 + 4 * l;
  }
  // head h: q, then k, then v
  float4 x0[U], x1[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i;
    x0[i] = x1[i] = make_float4(0, 0, 0, 0);
    if (h < H) {
      const X* src = h < a.Hq ? static_cast<const X*>(a.q) + tok * a.q_stride + static_cast<int64_t>(h) * D
                     : h < a.Hq + Hkv
                         ? static_cast<const X*>(a.k) + tok * a.k_stride + static_cast<int64_t>(h - a.Hq) * D
                         : static_cast<const X*>(a.v) + tok * a.v_stride + static_cast<int64_t>(h - a.Hq - Hkv) * D;
      x0[i] = load4(src + e0);
      x1[i] = load4(src + e1);
    }
  }
  const int pos = max(__ldg(a.seq_lens + b), 0) - a.T + t;  // below 0, whatever the length: all padding
  bool ok = pos >= 0;
  if (ok && rot > 0 && pos >= a.rope.n_positions) {
    if (l == 0) record_error(a.err, DEV_ERR_POSITION);
    ok = false;
  }
  int page = -1;
  float4 c = make_float4(1, 1, 1, 1), s = make_float4(0, 0, 0, 0);
  if (ok) {
    const int64_t pi = pos >> a.page_shift;
    if (pi < a.max_pages) page = __ldg(a.page_table + b * a.max_pages + pi);
    if (l < rl) {
      const float* cs = a.rope.cos_sin + static_cast<int64_t>(pos) * rot + 4 * l;
      c = load4(cs);
      s = load4(cs + rot / 2);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i;
    const bool isq = h < a.Hq, isk = !isq && h < a.Hq + Hkv;
    const float* nw = isq ? a.rope.q_norm : isk ? a.rope.k_norm : nullptr;
    float ss = sq4(x0[i]) + sq4(x1[i]);
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (nw) {
      const float f = rsqrtf(ss * (1.0f / D) + a.rope.eps);
      x0[i] = scale4(x0[i], f, load4(nw + e0), a.rope.norm_offset);
      x1[i] = scale4(x1[i], f, load4(nw + e1), a.rope.norm_offset);
    }
    if ((isq || isk) && l < rl && ok) {
      const float4 p = x0[i], q = x1[i];
      if (a.rope.interleaved) {  // pairs (p.x, p.y), (p.z, p.w), (q.x, q.y), (q.z, q.w)
        x0[i] = make_float4(p.x * c.x - p.y * s.x, p.y * c.x + p.x * s.x, p.z * c.y - p.w * s.y, p.w * c.y + p.z * s.y);
        x1[i] = make_float4(q.x * c.z - q.y * s.z, q.y * c.z + q.x * s.z, q.z * c.w - q.w * s.w, q.w * c.w + q.z * s.w);
      } else {
        x0[i] = make_float4(p.x * c.x - q.x * s.x, p.y * c.y - q.y * s.y, p.z * c.z - q.z * s.z, p.w * c.w - q.w * s.w);
        x1[i] = make_float4(q.x * c.x + p.x * s.x, q.y * c.y + p.y * s.y, q.z * c.z + p.z * s.z, q.w * c.w + p.w * s.w);
      }
    }
    if (h >= H) continue;
    if (isq) {
      if (!ok) x0[i] = x1[i] = make_float4(0, 0, 0, 0);
      O* dst = static_cast<O*>(a.q_out) + (static_cast<int64_t>(tok) * a.Hq + h) * D;
      store4(dst + e0, x0[i]);
      store4(dst + e1, x1[i]);
    } else if (ok) {
      if (page < 0 || page >= a.c.n_pages) {
        if (l == 0) record_error(a.err, DEV_ERR_PAGE);
        continue;
      }
      const int hk = isk ? h - a.Hq : h - a.Hq - Hkv;
      C* dst = static_cast<C*>(isk ? a.c.k : a.c.v) + page * a.c.page_stride +
               (pos & (a.c.page_size - 1)) * a.c.slot_stride + hk * a.c.head_stride;
      const float sc = isk ? a.c.k_scale : a.c.v_scale;
      if (sc != 1.0f) {
        x0[i] = make_float4(x0[i].x / sc, x0[i].y / sc, x0[i].z / sc, x0[i].w / sc);
        x1[i] = make_float4(x1[i].x / sc, x1[i].y / sc, x1[i].z / sc, x1[i].w / sc);
      }
      store4(dst + e0, x0[i]);
      store4(dst + e1, x1[i]);
    }
  }
}

template <class X, class O, class C, int LG>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t st) {
  constexpr int NG = ATH / LG;
  const int H = a.Hq + 2 * a.c.n_kv_heads;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.T;
  // several heads per group once that still fills the device (8 CTAs per SM)
  const int64_t few = (tokens * ((H + ROWS - 1) / ROWS) + NG - 1) / NG, one = (tokens * H + NG - 1) / NG;
  if (few >= 8 * num_sms())
    return launch_pdl(append_kernel<X, O, C, LG, ROWS>, dim3(static_cast<unsigned>(few)), dim3(ATH), 0, st, a);
  return launch_pdl(append_kernel<X, O, C, LG, 1>, dim3(static_cast<unsigned>(one)), dim3(ATH), 0, st, a);
}

template <class X, class O, class C>
cudaError_t launch_dim(const AppendArgs& a, cudaStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch_d<X, O, C, 8>(a, st);
    case 128: return launch_d<X, O, C, 16>(a, st);
    default: return launch_d<X, O, C, 32>(a, st);
  }
}
template <class X, class O>
cudaError_t launch_c(const AppendArgs& a, cudaStream_t st) {
  return a.c.dtype == KQ_BF16 ? launch_dim<X, O, __nv_bfloat16>(a, st) : launch_dim<X, O, __nv_fp8_e4m3>(a, st);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int x_bf16, int out_bf16, cudaStream_t st) {
  if (x_bf16) return out_bf16 ? launch_c<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_c<__nv_bfloat16, float>(a, st);
  return out_bf16 ? launch_c<float, __nv_bfloat16>(a, st) : launch_c<float, float>(a, st);
}

}  // namespace kq
