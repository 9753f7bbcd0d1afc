// kq_join.cuh -- the second launch of the attention calls that leave split
// items in parts: the parts of an item joined in their ranges' order,
//   o = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k,
// by as many blocks as there are rows to join.  (A join by the last CTA to
// arrive needs no second launch, but reads an item's parts through one SM: a tree
// of 16 tokens on 8 heads of 128, 64 rows each over 1000 positions, took 30 us
// that way, of which 11 are what a single tile takes.)
//
// Bound: the parts are read once, from L2, and by chains of few loads: a block's
// threads read all parts' statistics at once, and eight vectors of sums are in
// flight per lane.  A warp takes 128 dims of a row of an item; with MANY parts
// expected, a block does, its eight warps sharing the parts.  With more items than
// ranges the blocks go by ranges, as each leaves one item at most to the next ones.
#pragma once

#include "kq_attn_kernel.cuh"

namespace kq {
namespace attn {


struct JoinParams {
  AttnArgs a;
  const Split* split;
  const float *part_ml, *part;  // [slots][rows] maximum and weight sum, [slots][rows][D]
  int RT, rows;                 // row tiles per head, rows of one
  int by_item;                  // split [items], else [ranges]
  float scale;                  // of the values
};

constexpr int JTH = 256, JOIN_MOST = 512;  // threads; ranges

template <int D, class Out, bool MANY>
__global__ void __launch_bounds__(JTH) join_kernel(const __grid_constant__ JoinParams p) {
  constexpr int JW = JTH / 32, X = D < 128 ? D / 4 : 32, NC = D / 4 / X;  // vectors of a chunk (a lane's each), chunks of a row
  __shared__ float factor[MANY ? 1 : JW][JOIN_MOST];
  __shared__ float4 sums[MANY ? JW : 1][MANY ? 32 : 1];
  __shared__ float total[MANY ? 2 * JW : 1];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 s4 = __ldcg(reinterpret_cast<const int4*>(p.split) + blockIdx.x);
  const Split sp = {s4.x, s4.y, s4.z, s4.w};
  if (sp.parts == 0) return;
  const int HR = p.a.c.n_kv_heads * p.RT, b = sp.item / HR, hr = sp.item - b * HR;
  const int hk = hr / p.RT, row0 = (hr - hk * p.RT) * p.rows, R = min(p.rows, p.a.T * p.a.G - row0);
  const int unit = MANY ? blockIdx.y : blockIdx.y * JW + warp, r = unit / NC, x0 = unit % NC * X;
  if (r >= R) return;  // (MANY: all of the block)
  auto slot_of = [&](int k) { return k == 0 ? sp.slot : 2 * (sp.range + k) + 1; };
  auto stat = [&](int k) { return __ldcg(reinterpret_cast<const float2*>(p.part_ml + (static_cast<int64_t>(slot_of(k)) * p.rows + r) * 2)); };
  // the parts' statistics, two per thread (MANY) or lane: others, of more parts, are read again
  const int me = MANY ? threadIdx.x : lane, all = MANY ? JTH : 32;
  float* e = factor[MANY ? 0 : warp];
  const float2 none = make_float2(-INFINITY, 0.0f), x1 = me < sp.parts ? stat(me) : none, x2 = me + all < sp.parts ? stat(me + all) : none;
  float mm = fmaxf(x1.x, x2.x);
  for (int k = me + 2 * all; k < sp.parts; k += all) mm = fmaxf(mm, stat(k).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
  if constexpr (MANY) {
    if (lane == 0) total[warp] = mm;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < JW; ++k) mm = fmaxf(mm, total[k]);
  }
  const float ms = mm == -INFINITY ? 0.0f : mm;
  float ll = 0.0f;
  for (int k = me; k < sp.parts; k += all) {
    const float2 x = k == me ? x1 : k == me + all ? x2 : stat(k);
    const float f = ex2(x.x - ms);
    e[k] = f;
    ll += f * x.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, o);
  if constexpr (MANY) {
    if (lane == 0) total[JW + warp] = ll;
    __syncthreads();
    ll = total[JW];
#pragma unroll
    for (int k = 1; k < JW; ++k) ll += total[JW + k];
  } else {
    __syncwarp();
  }
  float4 acc = make_float4(0, 0, 0, 0);
  constexpr int STEP = MANY ? JW : 1, FLY = 8;
  for (int k0 = MANY ? warp : 0; k0 < sp.parts; k0 += FLY * STEP) {
    float4 v[FLY];
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int k = k0 + i * STEP;
      v[i] = make_float4(0, 0, 0, 0);
      if (k < sp.parts && lane < X)
        v[i] = __ldcg(reinterpret_cast<const float4*>(p.part + (static_cast<int64_t>(slot_of(k)) * p.rows + r) * D) + x0 + lane);
    }
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int k = k0 + i * STEP;
      if (k < sp.parts) add4(acc, e[k], v[i]);
    }
  }
  if constexpr (MANY) {
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 1; k < JW; ++k) add4(acc, 1.0f, sums[k][lane]);
  }
  const float inv = ll == 0.0f ? 0.0f : p.scale / ll;
  const int row = row0 + r, t = row / p.a.G, h = hk * p.a.G + row - t * p.a.G;
  if (lane < X) put4(static_cast<Out*>(p.a.out) + ((static_cast<int64_t>(b) * p.a.T + t) * p.a.Hq + h) * D + 4 * (x0 + lane), acc, inv);
}

// ranges: of the first launch.
template <int D, class Out>
cudaError_t launch_join(const JoinParams& p, int ranges, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(p.a.B) * p.a.c.n_kv_heads * p.RT;
  const unsigned blocks = p.by_item ? static_cast<unsigned>(items) : ranges;
  const int units = (p.rows < p.a.T * p.a.G ? p.rows : p.a.T * p.a.G) * (D < 128 ? 1 : D / 128);
  if (items * 8 <= ranges) return launch_pdl(join_kernel<D, Out, true>, dim3(blocks, units), dim3(JTH), 0, st, p);
  return launch_pdl(join_kernel<D, Out, false>, dim3(blocks, (units + 7) / 8), dim3(JTH), 0, st, p);
}

}  // namespace attn
}  // namespace kq
