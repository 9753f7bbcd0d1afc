// kq_attn_wide.cu -- attention of verify blocks: more than 16 query rows (new
// tokens x heads of a group) per key-value head, bf16 queries and cache, heads
// of 64 or 128 values.  The same line of tiles, cut and joins as
// kq_attn_kernel.cuh; per tile of 64 positions, on the 5th-generation tensor
// cores with up to 128 rows as the M:
//   S = q K^T        (A: q in tensor memory, B: K rows in shared memory)
//   o += P V         (A: P = 2^(s - m) in tensor memory, B: V rows, N-major)
//
// Bound: with 32 rows and more the products of mma instructions cost more
// than the bytes (8 x 16 tokens x 4 heads over 6007 positions: 26 us of their
// pipe alone and 88 us in all, against 24 us for the bytes); tcgen05 has three
// times their rate.  One CTA per SM:
//  * four loader warps copy 16 positions each per tile into a ring of stages,
//    16 bytes at a time to where the matrix descriptors want them: cores of 8
//    positions x 8 dims, 128 bytes each, 144 apart along the dims so that a
//    warp's copies spread over the banks.  K is K-major and V, in the same
//    layout, N-major, so neither is transposed;
//  * one thread issues the products: S of the next tile before P V of this one;
//  * four softmax warps, a thread per row: the row's 64 scores come from tensor
//    memory, its weights go back as two bf16 parts (2^-17), as A operand.  A
//    row's maximum is raised, and its sums in tensor memory scaled down, only
//    when it grows by more than 2^8 (the weights stay below 2^8 and the sums
//    exact); warps without rows pass.
// Every wait is bounded: one that gives up sets the device error word, after
// which the CTA's roles run through without waiting.
//
// Values that some rows see and others do not: as in kq_attn_kernel.cuh a
// segment whose sums are not all finite runs again; the loaders then put zeros
// in the place of values that are not finite, and each row's thread adds those
// it sees from memory.
#include "kq_attn_kernel.cuh"

namespace kq {
namespace attn {
namespace {

constexpr int WTH = 9 * 32;     // softmax warps 0-3, loaders 4-7, products 8
constexpr int WSTART = 6;       // tiles' time that an item costs besides its tiles
constexpr int LC = 144;         // bytes between cores along the dims
constexpr float kGrow = 8.0f;   // log2 units that a row's maximum may lag behind
// tensor memory columns: q, S x 2, P x 2 (high parts, low parts), o
constexpr int CQ = 0, CS = 64, CP = 192, CO = 320, COLS = 512;

template <int D>
struct WCfg {
  static constexpr int LR = D / 8 * LC;        // bytes between cores along the positions
  static constexpr int TILE = TK / 8 * LR;     // K or V of a tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int S = D == 128 ? 5 : 8;   // stages
  static constexpr int LAG = 2;                // tiles whose copies are in flight behind the newest
  static constexpr int SMEM = S * STAGE;
};

struct Bars {
  uint64_t full[8], empty[8], s_full[2], p_full[2], pv_done[2], q_full;
  uint32_t tmem;
  int bad, last;
  int scan[NW];
  float s_i[kWideRows];
};

__device__ __forceinline__ uint64_t core_desc(uint32_t saddr, uint32_t k_step, uint32_t n_step) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>((k_step >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>((n_step >> 4) & 0x3FFF) << 32) | (static_cast<uint64_t>(1) << 46);
}
// kind::f16, fp32 accumulator, bf16 operands, M = 128; n_major: B's N is contiguous
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// After the wait for tensor-memory loads: uses of v stay behind it.
__device__ __forceinline__ void tie(uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D>
struct Wide {
  using W = WCfg<D>;
  const Params& p;
  const Seg& g;
  Bars& bars;
  uint8_t* ring;
  uint32_t tb;   // tensor memory
  int tile0;     // tiles of earlier segments: the barriers' phases and the ring go on
  bool ok;       // no wait has given up

  __device__ __forceinline__ void wait(uint64_t* bar, int phase) {
    if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, static_cast<uint32_t>(phase & 1), p.a.err));
  }

  // ---- loaders: 16 positions of each tile
  template <bool CAREFUL>
  __device__ __forceinline__ void load(int lw, int lane) {
    const int n = g.t1 - g.t0, b0 = g.t0 * TK + lw * WT;
    auto page_of = [&](int base) {
      const int j = base + (lane & 15);
      return j >= g.first && j < g.len ? __ldg(g.table + (j >> p.a.page_shift)) : 0;
    };
    int page = page_of(b0);
    for (int i = 0; i < n + W::LAG; ++i) {
      if (i < n) {
        const int gi = tile0 + i, st = gi % W::S;
        const int next = i + 1 < n ? page_of(b0 + (i + 1) * TK) : 0;
        if (gi >= W::S) wait(&bars.empty[st], gi / W::S - 1);
        if (ok) copy(smem_u32(ring) + st * W::STAGE + 2 * lw * W::LR, b0 + i * TK, page, lane);
        page = next;
      }
      copy_commit();
      if (i >= W::LAG) {
        const int gi = tile0 + i - W::LAG, st = gi % W::S;
        copy_wait<W::LAG>();
        if constexpr (CAREFUL) {
          __syncwarp();
          for (int x = lane; x < WT * D; x += 32) {
            const int r = x / D, d = x % D;
            auto* v = reinterpret_cast<__nv_bfloat16*>(ring + st * W::STAGE + W::TILE + (2 * lw + r / 8) * W::LR + d / 8 * LC +
                                                       r % 8 * 16 + d % 8 * 2);
            if (!finite(__bfloat162float(*v))) *v = __float2bfloat16_rn(0.0f);
          }
        }
        fence_proxy_async_smem();  // the copies, seen by the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.full[st]);
      }
    }
    copy_wait<0>();
  }
  __device__ __forceinline__ void copy(uint32_t dst, int base, int page, int lane) {
    const AttnArgs& a = p.a;
    constexpr int CH = D / 8;  // 16-byte chunks per row
    if (base >= g.first && base + WT <= g.len && a.c.page_size >= WT / 2 &&
        __all_sync(0xFFFFFFFFu, static_cast<unsigned>(page) < a.c.n_pages)) {
      const int64_t row = a.c.slot_stride * 2;  // bytes
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pg = __shfl_sync(0xFFFFFFFFu, page, 8 * h);
        int64_t src = (pg * a.c.page_stride + g.head_off) * 2 + (((base + 8 * h) & (a.c.page_size - 1)) + lane / CH) * row +
                      lane % CH * 16;
        uint32_t to = dst + h * W::LR + lane % CH * LC + lane / CH * 16;
#pragma unroll
        for (int i = 0; i < CH / 4; ++i) {
          copy16(to, static_cast<const uint8_t*>(a.c.k) + src, true);
          copy16(to + W::TILE, static_cast<const uint8_t*>(a.c.v) + src, true);
          src += 32 / CH * row;
          to += 32 / CH * 16;
        }
      }
    } else {
      copy_rows(dst, base, page, lane);
    }
  }
  __device__ __noinline__ void copy_rows(uint32_t dst, int base, int page, int lane) {
    const AttnArgs& a = p.a;
    constexpr int CH = D / 8;
    const int64_t off = offset_of(base + (lane & 15), page);
#pragma unroll 1
    for (int i = 0; i < CH / 2; ++i) {
      const int c = i * 32 + lane, row = c / CH, col = c % CH;
      const int64_t ro = __shfl_sync(0xFFFFFFFFu, off, row);
      const bool on = ro >= 0;
      const int64_t src = (on ? ro : 0) + col * 16;
      const uint32_t to = dst + row / 8 * W::LR + col * LC + row % 8 * 16;
      copy16(to, static_cast<const uint8_t*>(a.c.k) + src, on);
      copy16(to + W::TILE, static_cast<const uint8_t*>(a.c.v) + src, on);
    }
  }
  // Bytes from the pool's start to position j's row; -1 where none is to be read.
  __device__ __forceinline__ int64_t offset_of(int j, int page) const {
    const AttnArgs& a = p.a;
    if (j < g.first || j >= g.len) return -1;
    if (page < 0 || page >= a.c.n_pages) {
      record_error(a.err, DEV_ERR_PAGE);
      return -1;
    }
    return (page * a.c.page_stride + (j & (a.c.page_size - 1)) * a.c.slot_stride + g.head_off) * 2;
  }

  // ---- products, by one warp (its first lane issues)
  __device__ __forceinline__ void products(int lane, int segment) {
    const int n = g.t1 - g.t0;
    const uint32_t rs = smem_u32(ring);
    wait(&bars.q_full, segment);
    auto scores = [&](int gi) {
      wait(&bars.full[gi % W::S], gi / W::S);
      tc_fence_after();
      if (lane == 0) {
        const uint32_t k = rs + gi % W::S * W::STAGE;
        if (ok)
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            tc_mma_ts(tb + CS + 64 * (gi & 1), tb + CQ + 8 * i, core_desc(k + i * 2 * LC, LC, W::LR), idesc(TK, false), i > 0);
        tc_commit(&bars.s_full[gi & 1]);
      }
      __syncwarp();
    };
    scores(tile0);
    for (int i = 0; i < n; ++i) {
      const int gi = tile0 + i;
      if (i + 1 < n) scores(gi + 1);  // S of that half was read before P of tile gi - 1 was ready
      wait(&bars.p_full[gi & 1], gi >> 1);
      tc_fence_after();
      if (lane == 0) {
        const uint32_t v = rs + gi % W::S * W::STAGE + W::TILE;
        if (ok)
#pragma unroll
          for (int k = 0; k < TK / 16; ++k)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              tc_mma_ts(tb + CO, tb + CP + 64 * (gi & 1) + 32 * t + 8 * k, core_desc(v + k * 2 * W::LR, W::LR, LC), idesc(D, true),
                        i > 0 || k > 0 || t > 0);
        tc_commit(&bars.pv_done[gi & 1]);
        tc_commit(&bars.empty[gi % W::S]);
      }
      __syncwarp();
    }
  }

  // ---- softmax: a thread per row
  float m, l;
  __device__ __forceinline__ void load_q(const __nv_bfloat16* src, uint32_t lanes, bool active) {
    if (active) {
#pragma unroll
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = src ? __ldg(reinterpret_cast<const uint4*>(src + 2 * c) + i) : make_uint4(0, 0, 0, 0);
          v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        }
        tmem_st16(tb + lanes + CQ + c, v);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.q_full);
  }
  // Scales the row's sums in tensor memory by c.
  __device__ __noinline__ void scale_sums(uint32_t lanes, float c) {
#pragma unroll 1
    for (int d = 0; d < D; d += 16) {
      uint32_t v[16];
      tmem_ld16(tb + lanes + CO + d, v);
      tmem_wait_ld();
      tie(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * c);
      tmem_st16(tb + lanes + CO + d, v);
    }
    tmem_wait_st();
  }
  // f: from the raw product to log2 units, or to the cap's argument; extra [D]: what the careful run adds.
  template <bool CAREFUL>
  __device__ __forceinline__ void softmax(uint32_t lanes, bool active, int pos, float f, float* extra) {
    const AttnArgs& a = p.a;
    const int n = g.t1 - g.t0;
    const int all_lo = a.window > 0 ? g.len - a.window : 0, all_hi = g.len - a.T;
    m = -INFINITY;
    l = 0.0f;
    for (int i = 0; i < n; ++i) {
      const int gi = tile0 + i, buf = gi & 1, base = (g.t0 + i) * TK;
      wait(&bars.s_full[buf], gi >> 1);
      tc_fence_after();
      if (active) {
        float s[TK];
        {
          uint32_t v[4][16];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld16(tb + lanes + CS + 64 * buf + 16 * c, v[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tie(v[c]);
#pragma unroll
            for (int e = 0; e < 16; ++e) s[16 * c + e] = __uint_as_float(v[c][e]);
          }
        }
        // the raw products are scaled inside the exponent; a cap, or a factor that turns the order around, comes first
        float scale = f;
        if (a.softcap > 0.0f || !(f > 0.0f)) {
          scale = 1.0f;
#pragma unroll
          for (int e = 0; e < TK; ++e) s[e] = a.softcap > 0.0f ? a.softcap * 1.4426950408889634f * tanhf(s[e] * f) : s[e] * f;
        }
        if (base < all_lo || base + TK - 1 > all_hi) {
#pragma unroll
          for (int e = 0; e < TK; ++e)
            if (!(base + e <= pos && (a.window == 0 || base + e > pos - a.window))) s[e] = -INFINITY;
        }
        float top[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = s[e];
#pragma unroll
        for (int e = 4; e < TK; ++e) top[e & 3] = fmaxf(top[e & 3], s[e]);
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
        const bool grow = mx > (m == -INFINITY ? m : m + kGrow);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float c = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2(m - mx);
          if (grow) m = mx;
          l *= c;
          if (i > 0) {
            wait(&bars.pv_done[buf ^ 1], (gi - 1) >> 1);
            tc_fence_after();
            scale_sums(lanes, c);
          }
        }
        const float mm = m == -INFINITY ? 0.0f : m;  // nothing seen yet: the weights are 0
        const float2 sc = make_float2(scale, scale), off = make_float2(-mm, -mm);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int e = 0; e < TK; e += 2) {
          const float2 x = ffma2(make_float2(s[e], s[e + 1]), sc, off);
          s[e] = ex2(x.x);
          s[e + 1] = ex2(x.y);
          sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], make_float2(s[e], s[e + 1]));
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if constexpr (CAREFUL) add_bad(base, pos, s, extra);
        if (gi >= 2) wait(&bars.pv_done[buf], (gi - 2) >> 1);  // P of two tiles ago is used up
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = make_float2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]);
            hi[e] = pack2<false>(x.x, x.y);
            const float2 b = unpack2<false>(hi[e]), d = fadd2(x, make_float2(-b.x, -b.y));
            lo[e] = pack2<false>(d.x, d.y);
          }
          tmem_st16(tb + lanes + CP + 64 * buf + 16 * c, hi);
          tmem_st16(tb + lanes + CP + 64 * buf + 32 + 16 * c, lo);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.p_full[buf]);
    }
    const int last = tile0 + n - 1;
    wait(&bars.pv_done[last & 1], last >> 1);
    tc_fence_after();
  }
  // The values of a tile that are not finite, to the row's extra sums if it sees them (weights w).
  __device__ __noinline__ void add_bad(int base, int pos, const float (&w)[TK], float* extra) {
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    for (int e = 0; e < TK; ++e) {
      const int j = base + e;
      const int page = j >= g.first && j < g.len ? __ldg(g.table + (j >> a.page_shift)) : 0;
      const int64_t off = offset_of(j, page);  // the same in every lane
      if (off < 0) continue;
      const auto* v = reinterpret_cast<const __nv_bfloat16*>(static_cast<const uint8_t*>(a.c.v) + off);
      bool bad = false;
      for (int d = lane; d < D; d += 32) bad |= !finite(__bfloat162float(v[d]));
      if (!__any_sync(0xFFFFFFFFu, bad)) continue;
      const bool sees = j <= pos && (a.window == 0 || j > pos - a.window);
      for (int d = 0; d < D; ++d) {
        const float x = __bfloat162float(v[d]);
        if (sees && !finite(x)) extra[d] += w[e] * x;
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(WTH, 1) wide_kernel(const __grid_constant__ Params p) {
  using W = WCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Bars bars;
  __shared__ __align__(16) float s_sum[JOIN_SUMS];
  const AttnArgs& a = p.a;
  uint8_t* ring = smem;
  int* prefix = reinterpret_cast<int*>(ring + W::S * W::STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < W::S; ++i) { mbar_init(&bars.full[i], 4); mbar_init(&bars.empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&bars.s_full[i], 1); mbar_init(&bars.p_full[i], 4); mbar_init(&bars.pv_done[i], 1); }
    mbar_init(&bars.q_full, 4);
    fence_mbar_init();
  }
  if (warp == 8) { tmem_alloc(&bars.tmem, COLS); tmem_relinquish(); }
  pdl_wait();
  pdl_launch_dependents();
  build_prefix(a, WSTART, prefix, bars.scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = bars.tmem;
  const Line line(a, p.RT, prefix);
  const int range = blockIdx.x;
  const int lo = line.bound(min(range, line.nc)), hi = range < line.nc ? line.bound(range + 1) : lo;
  int tile0 = 0, segment = 0;
  bool ok = true;
  for (int u = lo; u < hi;) {
    const Item it(a, line, p.RT, WSTART, u);
    const int end = min(it.i1, hi);
    if (u < it.i0) u = it.i0;
    if (u >= end) {  // none of its tiles is in this range
      u = end;
      continue;
    }
    const int r0 = it.rt * kWideRows, R = min(kWideRows, a.T * a.G - r0);
    const int r = threadIdx.x, row = min(r0 + r, a.T * a.G - 1), t = row / a.G, h = it.hk * a.G + row - t * a.G;  // warps 0-3
    auto out_row = [&](int rr) {
      const int x = r0 + rr, tt = x / a.G, hh = it.hk * a.G + x - tt * a.G;
      return static_cast<__nv_bfloat16*>(a.out) + ((static_cast<int64_t>(it.b) * a.T + tt) * a.Hq + hh) * D;
    };
    if (it.len == 0) {
      for (int x = threadIdx.x; x < R * (D / 4); x += WTH) put4(out_row(x / (D / 4)) + 4 * (x % (D / 4)), make_float4(0, 0, 0, 0), 0.0f);
      u = end;
      continue;
    }
    Seg g;
    g.len = it.len;
    g.first = first_of(a, it.len);
    g.table = a.page_table + it.b * a.max_pages;
    g.head_off = it.hk * a.c.head_stride;
    g.t0 = u - it.i0 + g.first / TK;
    g.t1 = end - it.i0 + g.first / TK;
    if (threadIdx.x == 0) bars.bad = 0;
    __syncthreads();  // the ring, the sums and tensor memory are free

    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const bool active = warp < 4 && 32 * warp < R;
    const float f = a.scale * a.c.k_scale * (a.softcap > 0.0f ? 1.0f / a.softcap : 1.4426950408889634f);
    Wide<D> w{p, g, bars, ring, tb, tile0, ok, -INFINITY, 0.0f};
    float extra[D];
    bool careful = false;
    for (;;) {
      if (warp < 4) {
        const auto* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(it.b) * a.T + t) * a.q_stride + static_cast<int64_t>(h) * D;
        w.load_q(r < R ? q : nullptr, lanes, active);
        const int pos = it.len - a.T + t;
        if (!careful) {
          w.template softmax<false>(lanes, active, pos, f, nullptr);
          if (active) {
            bool bad = false;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
              uint32_t v[16];
              tmem_ld16(tb + lanes + CO + d, v);
              tmem_wait_ld();
              tie(v);
#pragma unroll
              for (int i = 0; i < 16; ++i) bad |= !finite(__uint_as_float(v[i]));
            }
            if (bad && r < R) bars.bad = 1;
          }
        } else {
          for (int d = 0; d < D; ++d) extra[d] = 0.0f;
          w.template softmax<true>(lanes, active, pos, f, extra);
        }
      } else if (warp < 8) {
        if (careful) w.template load<true>(warp - 4, lane);
        else w.template load<false>(warp - 4, lane);
      } else {
        w.products(lane, segment);
      }
      ++segment;
      w.tile0 += g.t1 - g.t0;
      __syncthreads();
      if (careful || !bars.bad) break;
      careful = true;
      __syncthreads();
    }
    tile0 = w.tile0;
    ok = w.ok;

    const bool whole = u == it.i0 && end == it.i1;
    if (warp < 4) {
      const int slot = 2 * range + (lo >= it.i0 ? 1 : 0);  // the range starts in these tiles (1), or before them
      if (active) {
        const float inv = w.l == 0.0f ? 0.0f : a.c.v_scale / w.l;
        float* part = p.part + (static_cast<int64_t>(slot) * kWideRows + r) * D;
#pragma unroll 1
        for (int d = 0; d < D; d += 16) {
          uint32_t v[16];
          tmem_ld16(tb + lanes + CO + d, v);
          tmem_wait_ld();
          tie(v);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            float4 x = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            if (careful) x = make_float4(x.x + extra[d + i], x.y + extra[d + i + 1], x.z + extra[d + i + 2], x.w + extra[d + i + 3]);
            if (r < R) {
              if (whole) put4(out_row(r) + d + i, x, inv);
              else *reinterpret_cast<float4*>(part + d + i) = x;
            }
          }
        }
        if (!whole && r < R)
          *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(slot) * kWideRows + r) * 2) = make_float2(w.m, w.l);
      }
      tc_fence_before();
      if (!whole)
        join_parts<D, kWideRows>(p, line, it, R, threadIdx.x, reinterpret_cast<float*>(ring), W::S * W::STAGE, s_sum, bars.s_i, &bars.last,
                                 softmax_sync, [&](int rr, int d, float4 v, float inv) { put4(out_row(rr) + d, v, inv); });
    }
    u = end;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tb, COLS);
}

template <int D>
cudaError_t launch_d(const Params& p, cudaStream_t st) {
  using W = WCfg<D>;
  const size_t smem = W::SMEM + 4 * (static_cast<size_t>(p.a.B) + 1);
  static int set[64] = {0};
  const int dev = current_device_id();
  if (set[dev] < static_cast<int>(smem)) {
    const cudaError_t e = cudaFuncSetAttribute(wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    set[dev] = static_cast<int>(smem);
  }
  return launch_pdl(wide_kernel<D>, dim3(num_sms()), dim3(WTH), smem, st, p);
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_wide(const attn::Params& p, cudaStream_t st) {
  return p.a.c.head_dim == 64 ? attn::launch_d<64>(p, st) : attn::launch_d<128>(p, st);
}

}  // namespace kq
