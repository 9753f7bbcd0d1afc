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
// TREE: the position that a token is rotated by comes from its mask, its slot as
// before: 48 x 63 nodes of 48 heads of 128, bf16 into e4m3, 26 us (2.7 TB/s; 700
// instructions a warp, issued at 62%, and accesses of 4 and 8 bytes: neither by
// itself is the bound); 16 nodes 2.4 us.
#include "kq_cache.h"
#include "kq_vec.cuh"

namespace kq {
namespace {

constexpr int ATH = 128;  // threads per CTA
constexpr int ROWS = 3;   // rows per group of lanes at a time

// X: q, k, v; O: q_out; C: the cache.  LG = D / 8 lanes hold one row; U rows per group of lanes.
template <class X, class O, class C, int LG, int U, bool TREE>
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
  const int len = max(__ldg(a.seq_lens + b), 0);
  const int slot = len - a.T + t;  // below 0, whatever the length: all padding
  int pos = slot;
  if constexpr (TREE) pos = tree_position(tree_bits(__ldg(a.tree + tok), a.T, t, len), a.T, len);
  bool ok = pos >= 0;
  if (ok && rot > 0 && pos >= a.rope.n_positions) {
    if (l == 0) record_error(a.err, DEV_ERR_POSITION);
    ok = false;
  }
  int page = -1;
  float4 c = make_float4(1, 1, 1, 1), s = make_float4(0, 0, 0, 0);
  if (ok) {
    const int64_t pi = slot >> a.page_shift;
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
    if ((isq || isk) && l < rl && ok) rotate8(x0[i], x1[i], c, s, a.rope.interleaved);
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
               (slot & (a.c.page_size - 1)) * a.c.slot_stride + hk * a.c.head_stride;
      const float sc = isk ? a.c.k_scale : a.c.v_scale;
      if (sc != 1.0f) {
        x0[i] = over4(x0[i], sc);
        x1[i] = over4(x1[i], sc);
      }
      store4(dst + e0, x0[i]);
      store4(dst + e1, x1[i]);
    }
  }
}

template <class X, class O, class C, int LG, bool TREE>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t st) {
  constexpr int NG = ATH / LG;
  const int H = a.Hq + 2 * a.c.n_kv_heads;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.T;
  // several heads per group once that still fills the device (8 CTAs per SM)
  const int64_t few = (tokens * ((H + ROWS - 1) / ROWS) + NG - 1) / NG, one = (tokens * H + NG - 1) / NG;
  if (few >= 8 * num_sms())
    return launch_pdl(append_kernel<X, O, C, LG, ROWS, TREE>, dim3(static_cast<unsigned>(few)), dim3(ATH), 0, st, a);
  return launch_pdl(append_kernel<X, O, C, LG, 1, TREE>, dim3(static_cast<unsigned>(one)), dim3(ATH), 0, st, a);
}

template <class X, class O, class C, bool TREE>
cudaError_t launch_dim(const AppendArgs& a, cudaStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch_d<X, O, C, 8, TREE>(a, st);
    case 128: return launch_d<X, O, C, 16, TREE>(a, st);
    default: return launch_d<X, O, C, 32, TREE>(a, st);
  }
}
template <class X, class O>
cudaError_t launch_c(const AppendArgs& a, cudaStream_t st) {
  if (a.c.dtype == KQ_BF16) return a.tree ? launch_dim<X, O, __nv_bfloat16, true>(a, st) : launch_dim<X, O, __nv_bfloat16, false>(a, st);
  return a.tree ? launch_dim<X, O, __nv_fp8_e4m3, true>(a, st) : launch_dim<X, O, __nv_fp8_e4m3, false>(a, st);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs& a, int x_bf16, int out_bf16, cudaStream_t st) {
  if (x_bf16) return out_bf16 ? launch_c<__nv_bfloat16, __nv_bfloat16>(a, st) : launch_c<__nv_bfloat16, float>(a, st);
  return out_bf16 ? launch_c<float, __nv_bfloat16>(a, st) : launch_c<float, float>(a, st);
}

}  // namespace kq
