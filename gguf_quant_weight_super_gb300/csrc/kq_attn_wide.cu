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
// times their rate: 54 us here, of which the copies alone take 45 (7 us until
// the first tile is there, 10 us for the parts' join).  20 rows 49 us against
// 51 with mma, 128 rows 75 against 139.  Where the joins of 128-row parts outweigh
// that, with few heads, the host takes mma (kq_attn.cu).  One CTA per SM:
//  * seven loader warps copy 8 positions at a time into a ring of stages, 16
//    bytes per lane, where the matrix descriptors' 128-byte swizzle wants them:
//    64 dims of a position are a line of 128 bytes, its 16-byte chunks c at
//    c ^ (position & 7).  K is K-major and V, in the same layout, N-major, so
//    neither is transposed.  (Without swizzle, cores of 8 positions x 16 bytes,
//    each line takes pieces of eight rows, and the copies alone ran at 3.7
//    TB/s.)  A stage's barrier is told by the copies themselves as they land,
//    so that all stages (192 KB) can be in flight;
//  * one thread issues the products: S of the next tile before P V of this one;
//  * eight softmax warps, two threads per row, 32 positions each: the scores
//    come from tensor memory, the weights go back as two bf16 parts (2^-17), as
//    A operand.  One thread per row took 1.3 us a tile, twice the bytes' time.
//    A row's maximum is raised, and its sums in tensor memory scaled down, only
//    when it grows by more than 2^8 (the weights stay below 2^8 and the sums
//    exact); warps without rows pass.
// TREE: masks, and parts joined by a second launch, as in kq_attn_kernel.cuh; a
// row's maximum may lag by 2^24, since of 128 rows one grows by 2^8 in every
// fourth tile, and a scaling takes a tile's time (weights have bf16's range, their
// parts and sums fp32's).  8 x 61 nodes of 4 heads a group, 0 to 6007 positions, 8
// heads of 128: 72 us, of which the join is 8.
//
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

constexpr int NLOAD = 7;        // loader warps
constexpr int WTH = (8 + NLOAD + 1) * 32;  // softmax warps 0-7, loaders 8-14, products 15
constexpr int HC = TK / 2;      // a softmax thread's positions of a tile
constexpr int WSTART = 6;       // tiles' time that an item costs besides its tiles
// log2 units that a row's maximum may lag behind.  (Trees' blocks have up to 128 rows, of which with 8 units one grows often.)
template <bool TREE>
constexpr float kGrow = TREE ? 24.0f : 8.0f;
// tensor memory columns: q, S x 2, P x 2 (high parts, low parts), o
constexpr int CQ = 0, CS = 64, CP = 192, CO = 320, COLS = 512;

template <int D>
struct WCfg {
  static constexpr int HALF = TK * 128;        // 64 dims of a tile's positions
  static constexpr int TILE = D / 64 * HALF;   // K or V of a tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int S = D == 128 ? 6 : 12;  // stages
  static constexpr int SMEM = S * STAGE;
};

struct Bars {
  uint64_t full[12], empty[12], s_full[2], p_full[2], pv_done[2], q_full;
  uint32_t tmem;
  int bad, last;
  int scan[NW];
  float s_i[kWideRows];
  float top[2][2][kWideRows];  // tile parity, half: the rows' largest score; at the end their weight sums
};

// Shared-memory operand in 128-byte-swizzled groups of 8 lines (1024 bytes apart); mn_step: bytes from 64 values along M or
// N to the next (N-major operands).
__device__ __forceinline__ uint64_t line_desc(uint32_t saddr, uint32_t mn_step) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>((mn_step >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
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
__device__ __forceinline__ void first_half_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 2, 256;" ::: "memory"); }
// The two warps of 32 rows.
__device__ __forceinline__ void rows_sync(int quarter) { asm volatile("bar.sync %0, 64;" ::"r"(3 + quarter) : "memory"); }

// A row's place: its position and what it sees of a tree's tokens.
template <bool TREE>
struct Place {
  int pos;
  uint64_t bits;
};
template <>
struct Place<false> {
  int pos;
  static constexpr uint64_t bits = 0;
};

template <int D, bool TREE>
struct Wide {
  using W = WCfg<D>;
  const Params& p;
  const Seg g;
  Bars& bars;
  uint8_t* ring;
  uint32_t tb;   // tensor memory
  int tile0;     // tiles of earlier segments: the barriers' phases and the ring go on
  bool ok;       // no wait has given up

  __device__ __forceinline__ void wait(uint64_t* bar, int phase) {
    if (__all_sync(0xFFFFFFFFu, test(bar, phase & 1))) return;
    if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, static_cast<uint32_t>(phase & 1), p.a.err));
  }
  static __device__ __forceinline__ bool test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return done != 0;
  }

  // ---- loaders: 8 positions at a time, in turn
  template <bool CAREFUL>
  __device__ __forceinline__ void load(int lw, int lane) {
    const AttnArgs& a = p.a;
    const int n = g.t1 - g.t0, b0 = g.t0 * TK;
    auto page_of = [&](int x) {  // of this lane's row (lane & 7)
      const int j = b0 + 8 * x + (lane & 7);
      return j >= g.first && j < g.len ? __ldg(g.table + (j >> a.page_shift)) : 0;
    };
    int page = lw < 8 * n ? page_of(lw) : 0;
    for (int x = lw; x < 8 * n; x += NLOAD) {
      const int gi = tile0 + (x >> 3), st = gi % W::S, base = b0 + 8 * x;
      const int next = x + NLOAD < 8 * n ? page_of(x + NLOAD) : 0;
      if (gi >= W::S) wait(&bars.empty[st], gi / W::S - 1);
      uint8_t* lines = ring + st * W::STAGE + (x & 7) * 1024;
      const int64_t off = offset_of(p, g, base + (lane & 7), page);  // this lane's row's
      if (ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = (lane >> 3) + 4 * i;
          int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
          const bool on = src >= 0;
          src = (on ? src : 0) + (lane & 7) * 16;
          const uint32_t to = smem_u32(lines) + r * 128 + ((lane & 7) ^ r) * 16;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            copy16(to + h * W::HALF, static_cast<const uint8_t*>(a.c.k) + src + h * 128, on);
            copy16(to + h * W::HALF + W::TILE, static_cast<const uint8_t*>(a.c.v) + src + h * 128, on);
          }
        }
      }
      page = next;
      if constexpr (CAREFUL) {
        copy_commit();
        copy_wait<0>();
        __syncwarp();
        for (int y = lane; y < 8 * D; y += 32) {
          const int r = y / D, d = y % D;
          auto* v = reinterpret_cast<__nv_bfloat16*>(lines + W::TILE + d / 64 * W::HALF + r * 128 + ((d % 64 / 8) ^ r) * 16 + d % 8 * 2);
          if (!finite(__bfloat162float(*v))) *v = __float2bfloat16_rn(0.0f);
        }
        mbar_arrive(&bars.full[st]);
      } else {  // each thread's arrival, once its copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars.full[st])) : "memory");
      }
    }
    copy_commit();
    copy_wait<0>();
  }
  // Bytes from the pool's start to position j's row; -1 where none is to be read.
  static __device__ __forceinline__ int64_t offset_of(const Params& p, const Seg& g, int j, int page) {
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
      fence_proxy_async_smem();  // the copies, which the barrier has put before this, seen by the tensor cores
      tc_fence_after();
      if (lane == 0) {
        const uint32_t k = rs + gi % W::S * W::STAGE;
        if (ok)
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            tc_mma_ts(tb + CS + 64 * (gi & 1), tb + CQ + 8 * i, line_desc(k + i / 4 * W::HALF + i % 4 * 32, 16), idesc(TK, false), i > 0);
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
              tc_mma_ts(tb + CO, tb + CP + 64 * (gi & 1) + 32 * t + 8 * k, line_desc(v + k * 2048, W::HALF), idesc(D, true),
                        i > 0 || k > 0 || t > 0);
        tc_commit(&bars.pv_done[gi & 1]);
        tc_commit(&bars.empty[gi % W::S]);
      }
      __syncwarp();
    }
  }

  // ---- softmax: two threads per row, warps w and w + 4 (half 0, 1)
  float m, l;
  __device__ __forceinline__ void load_q(const __nv_bfloat16* src, uint32_t lanes, int half, bool active) {
    if (active) {
#pragma unroll
      for (int c = 0; c < D / 4; c += 16) {
        const int col = half * (D / 4) + c;
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = src ? __ldg(reinterpret_cast<const uint4*>(src + 2 * col) + i) : make_uint4(0, 0, 0, 0);
          v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        }
        tmem_st16(tb + lanes + CQ + col, v);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.q_full);
  }
  // Scales the row's sums in tensor memory, D / 2 of them from column `sums`, by c.
  static __device__ __noinline__ void scale_sums(uint32_t sums, float c) {
#pragma unroll 1
    for (int d = 0; d < D / 2; d += 16) {
      uint32_t v[16];
      tmem_ld16(sums + d, v);
      tmem_wait_ld();
      tie(v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * c);
      tmem_st16(sums + d, v);
    }
    tmem_wait_st();
  }
  // r: the row; f: from the raw product to log2 units, or to the cap's argument; extra [D]: what the careful run adds.
  template <bool CAREFUL>
  __device__ __forceinline__ void softmax(uint32_t lanes, int r, int half, bool active, Place<TREE> at, float f, float* extra) {
    const AttnArgs& a = p.a;
    const int n = g.t1 - g.t0;
    const int all_lo = a.window > 0 ? g.len - a.window : 0, all_hi = g.len - a.T - (TREE ? 1 : 0);
    m = TREE && at.pos < 0 ? INFINITY : -INFINITY;  // a tree's padding: weights of 0 wherever masks are not looked at
    l = 0.0f;
    for (int i = 0; i < n; ++i) {
      const int gi = tile0 + i, buf = gi & 1, tile = (g.t0 + i) * TK, base = tile + half * HC;
      wait(&bars.s_full[buf], gi >> 1);
      tc_fence_after();
      if (active) {
        float s[HC];
        {
          uint32_t v[2][16];
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld16(tb + lanes + CS + 64 * buf + HC * half + 16 * c, v[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
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
          for (int e = 0; e < HC; ++e) s[e] = a.softcap > 0.0f ? a.softcap * 1.4426950408889634f * tanhf(s[e] * f) : s[e] * f;
        }
        if (tile < all_lo || tile + TK - 1 > all_hi) {
#pragma unroll
          for (int e = 0; e < HC; ++e) {
            const int j = base + e;  // (a chain's test stands here itself: through sees(), 8 x 16 tokens took 55.0 us in place of 54.4)
            if (TREE ? !sees<TREE>(j, at.pos, at.bits, g.len - a.T, a.window) : !(j <= at.pos && (a.window == 0 || j > at.pos - a.window)))
              s[e] = -INFINITY;
          }
        }
        float top[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = s[e];
#pragma unroll
        for (int e = 4; e < HC; ++e) top[e & 3] = fmaxf(top[e & 3], s[e]);
        float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
        bars.top[buf][half][r] = mx;
        rows_sync(r >> 5);
        mx = fmaxf(mx, bars.top[buf][half ^ 1][r]);
        const bool grow = mx > (m == -INFINITY ? m : m + kGrow<TREE>);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float c = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2(m - mx);
          if (grow) m = mx;
          l *= c;
          if (i > 0) {
            wait(&bars.pv_done[buf ^ 1], (gi - 1) >> 1);
            tc_fence_after();
            scale_sums(tb + lanes + CO + half * (D / 2), c);
          }
        }
        const float mm = m == -INFINITY ? 0.0f : m;  // nothing seen yet: the weights are 0
        const float2 sc = make_float2(scale, scale), off = make_float2(-mm, -mm);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int e = 0; e < HC; e += 2) {
          const float2 x = ffma2(make_float2(s[e], s[e + 1]), sc, off);
          s[e] = ex2(x.x);
          s[e + 1] = ex2(x.y);
          sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], make_float2(s[e], s[e + 1]));
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if constexpr (CAREFUL) {
          float weights[HC];  // an array of its own: the call keeps it out of registers
#pragma unroll
          for (int e = 0; e < HC; ++e) weights[e] = s[e];
          add_bad(p, g, base, at, weights, extra);
        }
        // (P of two tiles ago, in the same columns, is used up: its product was issued before S of this tile)
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = make_float2(s[2 * e], s[2 * e + 1]);
          hi[e] = pack2<false>(x.x, x.y);
          const float2 b = unpack2<false>(hi[e]), d = fadd2(x, make_float2(-b.x, -b.y));
          lo[e] = pack2<false>(d.x, d.y);
        }
        tmem_st16(tb + lanes + CP + 64 * buf + 16 * half, hi);
        tmem_st16(tb + lanes + CP + 64 * buf + 32 + 16 * half, lo);
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
  // The values of a half tile that are not finite, to the row's extra sums if it sees them (weights w).
  static __device__ __noinline__ void add_bad(const Params& p, Seg g, int base, Place<TREE> at, const float* w, float* extra) {
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31;
    for (int e = 0; e < HC; ++e) {
      const int j = base + e;
      const int page = j >= g.first && j < g.len ? __ldg(g.table + (j >> a.page_shift)) : 0;
      const int64_t off = offset_of(p, g, j, page);  // the same in every lane
      if (off < 0) continue;
      const auto* v = reinterpret_cast<const __nv_bfloat16*>(static_cast<const uint8_t*>(a.c.v) + off);
      bool bad = false;
      for (int d = lane; d < D; d += 32) bad |= !finite(__bfloat162float(v[d]));
      if (!__any_sync(0xFFFFFFFFu, bad)) continue;
      const bool seen = sees<TREE>(j, at.pos, at.bits, g.len - a.T, a.window);
      for (int d = 0; d < D; ++d) {
        const float x = __bfloat162float(v[d]);
        if (seen && !finite(x)) extra[d] += w[e] * x;
      }
    }
  }
};

template <int D, bool TREE>
__global__ void __launch_bounds__(WTH, 1) wide_kernel(const __grid_constant__ Params p) {
  using W = WCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Bars bars;
  __shared__ __align__(16) float s_sum[JOIN_SUMS];
  const AttnArgs& a = p.a;
  uint8_t* ring = smem;
  int* prefix = reinterpret_cast<int*>(ring + W::S * W::STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < W::S; ++i) { mbar_init(&bars.full[i], 256); mbar_init(&bars.empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&bars.s_full[i], 1); mbar_init(&bars.p_full[i], 8); mbar_init(&bars.pv_done[i], 1); }
    mbar_init(&bars.q_full, 8);
    fence_mbar_init();
  }
  if (warp == 8 + NLOAD) { tmem_alloc(&bars.tmem, COLS); tmem_relinquish(); }
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
  if (TREE && threadIdx.x == 0 && !p.by_item) p.split[range].parts = 0;
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
    const int r = threadIdx.x & (kWideRows - 1), half = (warp >> 2) & 1;  // softmax warps
    const int row = min(r0 + r, a.T * a.G - 1), t = row / a.G, h = it.hk * a.G + row - t * a.G;
    auto out_row = [&](int rr) {
      const int x = r0 + rr, tt = x / a.G, hh = it.hk * a.G + x - tt * a.G;
      return static_cast<__nv_bfloat16*>(a.out) + ((static_cast<int64_t>(it.b) * a.T + tt) * a.Hq + hh) * D;
    };
    if (it.len == 0) {
      if (TREE && threadIdx.x == 0) note_split(p.split, p.by_item, line, it, range, true, 0);
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
    Place<TREE> at;
    if constexpr (TREE) {
      const TreeToken x(a, it.b, t, it.len);
      at = {x.pos, x.bits};
    } else {
      at.pos = it.len - a.T + t;
    }
    const bool padding = TREE && at.pos < 0;
    const bool active = warp < 8 && 32 * (warp & 3) < R;
    const float f = a.scale * a.c.k_scale * (a.softcap > 0.0f ? 1.0f / a.softcap : 1.4426950408889634f);
    Wide<D, TREE> w{p, g, bars, ring, tb, tile0, ok, -INFINITY, 0.0f};
    float extra[D];
    bool careful = false;
    for (;;) {
      if (warp < 8) {
        const auto* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(it.b) * a.T + t) * a.q_stride + static_cast<int64_t>(h) * D;
        w.load_q(r < R ? q : nullptr, lanes, half, active);
        if (!careful) {
          w.template softmax<false>(lanes, r, half, active, at, f, nullptr);
          if (active) {
            bool bad = false;
#pragma unroll 1
            for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 16) {
              uint32_t v[16];
              tmem_ld16(tb + lanes + CO + d, v);
              tmem_wait_ld();
              tie(v);
#pragma unroll
              for (int i = 0; i < 16; ++i) bad |= !finite(__uint_as_float(v[i]));
            }
            if (bad && r < R && !padding) bars.bad = 1;
          }
        } else {
          for (int d = 0; d < D; ++d) extra[d] = 0.0f;
          w.template softmax<true>(lanes, r, half, active, at, f, extra);
        }
        if (padding) {  // whatever the keys were
          w.m = -INFINITY;
          w.l = 0.0f;
        }
        bars.top[0][half][r] = w.l;  // read after the barrier
      } else if (warp < 8 + NLOAD) {
        if (careful) w.template load<true>(warp - 8, lane);
        else w.template load<false>(warp - 8, lane);
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
    if (TREE && u == it.i0 && threadIdx.x == 0) note_split(p.split, p.by_item, line, it, range, whole, 2 * range + (lo >= it.i0 ? 1 : 0));
    if (warp < 8) {
      const int slot = 2 * range + (lo >= it.i0 ? 1 : 0);  // the range starts in these tiles (1), or before them
      const float weight = bars.top[0][0][r] + bars.top[0][1][r];
      float* others = reinterpret_cast<float*>(ring);  // [2][rows][D]: what each half's positions add
      if (careful) {
        for (int d = 0; d < D; ++d) others[(half * kWideRows + r) * D + d] = extra[d];
        softmax_sync();
      }
      if (active) {
        const float inv = weight == 0.0f ? 0.0f : a.c.v_scale / weight;
        float* part = p.part + (static_cast<int64_t>(slot) * kWideRows + r) * D;
#pragma unroll 1
        for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 16) {
          uint32_t v[16];
          tmem_ld16(tb + lanes + CO + d, v);
          tmem_wait_ld();
          tie(v);
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            float4 x = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            if (careful)
              for (int e = 0; e < 2; ++e) add4(x, 1.0f, *reinterpret_cast<const float4*>(others + (e * kWideRows + r) * D + d + i));
            if (padding) x = make_float4(0, 0, 0, 0);
            if (r < R) {
              if (whole) put4(out_row(r) + d + i, x, inv);
              else *reinterpret_cast<float4*>(part + d + i) = x;
            }
          }
        }
        if (!whole && half == 0 && r < R)
          *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(slot) * kWideRows + r) * 2) = make_float2(w.m, weight);
      }
      tc_fence_before();
      if (!TREE && !whole) {
        softmax_sync();  // both halves' parts are stored
        if (half == 0)
          join_parts<D, kWideRows>(p, line, it, R, threadIdx.x, reinterpret_cast<float*>(ring), W::S * W::STAGE, s_sum, bars.s_i, &bars.last,
                                   first_half_sync, [&](int rr, int d, float4 v, float inv) { put4(out_row(rr) + d, v, inv); });
      }
    }
    u = end;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8 + NLOAD) tmem_dealloc(tb, COLS);
}

template <int D, bool TREE>
cudaError_t launch_d(const Params& p, cudaStream_t st, AttnShape* ask) {
  using W = WCfg<D>;
  const size_t smem = W::SMEM + 4 * (static_cast<size_t>(p.a.B) + 1);
  static bool set[64] = {false};
  const int dev = current_device_id();
  if (!set[dev]) {  // for all calls: one at the same time may want less
    constexpr int most = W::SMEM + 4 * (kMaxSeqs + 1);
    static_assert(most + 14 * 1024 <= kMaxSmemPerBlock, "beside the static memory");
    const cudaError_t e = cudaFuncSetAttribute(wide_kernel<D, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  if (ask) {
    ask->planned = 1;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ask->resident, wide_kernel<D, TREE>, WTH, smem);
  }
  const cudaError_t e = launch_pdl(wide_kernel<D, TREE>, dim3(num_sms()), dim3(WTH), smem, st, p);
  return !TREE || e != cudaSuccess ? e : launch_tree_join(p, kWideRows, D, false, num_sms(), st);
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_wide(const attn::Params& p, cudaStream_t st, AttnShape* ask) {
  if (p.a.tree) return p.a.c.head_dim == 64 ? attn::launch_d<64, true>(p, st, ask) : attn::launch_d<128, true>(p, st, ask);
  return p.a.c.head_dim == 64 ? attn::launch_d<64, false>(p, st, ask) : attn::launch_d<128, false>(p, st, ask);
}

}  // namespace kq
