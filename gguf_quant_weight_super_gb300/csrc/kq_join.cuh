// kq_join.cuh -- the second launch of the attention calls that leave split
// items in parts: the parts of an item joined in their ranges' order,
//   o = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k,
// by as many blocks as there are rows to join.  (A join by the last CTA to
// arrive needs no second launch, but reads an item's parts through one SM: a tree
// of 16 tokens on 8 heads of 128, 64 rows each over 1000 positions, took 30 us
// that way, of which 11 are what a single tile takes.)
//
// Bound: the parts are read once, from L2.  A block takes a range's item, eight
// rows of it, a warp each; or, with MANY parts expected, one row, whose parts its
// eight warps share.
#pragma once

#include "kq_attn_kernel.cuh"

namespace kq {
namespace attn {

// A range's item that goes on in the next ranges: the sequence, head * RT + row tile, the parts (0: none) and the first one's
// place.  The others lie at 2 * range + 1.
struct Split {
  int b, hr, parts, slot;
};

struct JoinParams {
  AttnArgs a;
  const Split* split;
  const float *part_ml, *part;  // [slots][rows] maximum and weight sum, [slots][rows][D]
  int RT, rows;                 // row tiles per head, rows of one
  float scale;                  // of the values
};

constexpr int JTH = 256, JOIN_MOST = 512;  // threads; ranges

template <int D, class Out, bool MANY>
__global__ void __launch_bounds__(JTH) join_kernel(const __grid_constant__ JoinParams p) {
  constexpr int JW = JTH / 32, X = D / 4, V = X < 32 ? 1 : X / 32;  // vectors of a row, and per lane
  __shared__ float factor[MANY ? 1 : JW][JOIN_MOST];
  __shared__ float4 sums[MANY ? JW : 1][MANY ? X : 1];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 s4 = __ldcg(reinterpret_cast<const int4*>(p.split) + blockIdx.x);
  const Split sp = {s4.x, s4.y, s4.z, s4.w};
  if (sp.parts == 0) return;
  const int hk = sp.hr / p.RT, row0 = (sp.hr - hk * p.RT) * p.rows, R = min(p.rows, p.a.T * p.a.G - row0);
  const int r = MANY ? blockIdx.y : blockIdx.y * JW + warp;
  if ((MANY ? r : r - warp) >= R) return;
  const bool on = r < R;
  auto slot_of = [&](int k) { return k == 0 ? sp.slot : 2 * (static_cast<int>(blockIdx.x) + k) + 1; };
  float* e = factor[MANY ? 0 : warp];
  float mm = -INFINITY, ll = 0.0f;
  if (on) {
    for (int k = lane; k < sp.parts; k += 32) mm = fmaxf(mm, __ldcg(p.part_ml + (static_cast<int64_t>(slot_of(k)) * p.rows + r) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
    const float ms = mm == -INFINITY ? 0.0f : mm;
    for (int k = lane; k < sp.parts; k += 32) {
      const float2 x = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (static_cast<int64_t>(slot_of(k)) * p.rows + r) * 2));
      const float f = ex2(x.x - ms);
      if (!MANY || warp == 0) e[k] = f;
      ll += f * x.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, o);
  }
  if (MANY) __syncthreads();
  else __syncwarp();
  float4 acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = make_float4(0, 0, 0, 0);
  if (on && lane < X) {
#pragma unroll 4
    for (int k = MANY ? warp : 0; k < sp.parts; k += MANY ? JW : 1) {
      const float4* part = reinterpret_cast<const float4*>(p.part + (static_cast<int64_t>(slot_of(k)) * p.rows + r) * D) + lane;
#pragma unroll
      for (int i = 0; i < V; ++i) add4(acc[i], e[k], __ldcg(part + 32 * i));
    }
  }
  const float inv = ll == 0.0f ? 0.0f : p.scale / ll;
  const int row = row0 + r, t = row / p.a.G, h = hk * p.a.G + row - t * p.a.G;
  Out* out = static_cast<Out*>(p.a.out) + ((static_cast<int64_t>(sp.b) * p.a.T + t) * p.a.Hq + h) * D;
  if constexpr (!MANY) {
    if (on && lane < X)
#pragma unroll
      for (int i = 0; i < V; ++i) put4(out + 4 * (lane + 32 * i), acc[i], inv);
  } else {
    if (lane < X)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    if (threadIdx.x < X) {
      float4 x = sums[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < JW; ++k) add4(x, 1.0f, sums[k][threadIdx.x]);
      put4(out + 4 * threadIdx.x, x, inv);
    }
  }
}

// ranges: of the first launch; items: (sequence, head, row tile).
template <int D, class Out>
cudaError_t launch_join(const JoinParams& p, int ranges, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(p.a.B) * p.a.c.n_kv_heads * p.RT;
  if (items * 8 <= ranges) return launch_pdl(join_kernel<D, Out, true>, dim3(ranges, p.rows), dim3(JTH), 0, st, p);
  return launch_pdl(join_kernel<D, Out, false>, dim3(ranges, (p.rows + 7) / 8), dim3(JTH), 0, st, p);
}

}  // namespace attn
}  // namespace kq
