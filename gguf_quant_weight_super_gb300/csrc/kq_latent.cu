// kq_latent.cu -- attention of the newest T tokens of each sequence over its
// cache of latent vectors c_j, which all heads share, in absorbed form:
//   s_j = scale q.c_j (latent and rope part),  o = sum_j softmax(s)_j c_j[0 .. C)
// in one pass with a running maximum and running sums, on the 5th-generation
// tensor cores, with up to 128 rows (tokens x heads) as the M.
//
// Bound: a vector of 1152 bytes (C = 512, bf16) serves 2 (2 C + 64) flops per
// row, with 128 rows 242 flops per byte, near the device's 282: bytes and
// products both have to run at their rate.  What is in the way is the room: the
// sums of 128 rows, 512 fp32 values each, are all of an SM's tensor memory, and
// the queries 144 KB of its shared memory.  So two SMs, a cluster, share 128 rows
// by halves of the latent's dims: each CTA keeps its half of q and of the sums in
// tensor memory, loads its half of every vector (the first also the rope part)
// and multiplies it once as keys and once as values,
//   S  = q_half K_half^T   (A: q in tensor memory; the rope part of q in shared memory)
//   o += P V_half          (A: P = 2^(s - m) in tensor memory; V: the same lines, N-major)
// Nothing is loaded or multiplied twice.  The price is S: each CTA has the sum
// over its half of the dims only, so the CTAs send each other their halves' sums
// (32 KB per tile of 64 positions and direction, straight from registers into the
// other's shared memory, which tells the barrier its bytes) and both go through
// the same softmax, bit for bit, as a + b is b + a.
//
// The roles of a CTA, as in kq_attn_wide.cu:
//  * loader warps copy 8 positions at a time into a ring of stages, 64 dims of a
//    position a line of 128 bytes in the matrix descriptors' 128-byte swizzle
//    (e4m3 becomes fp16 on the way, exactly);
//  * one warp issues S of the next tile and P V of this one, whichever can run;
//  * eight softmax warps, two threads per row, 32 positions each.  A tile's own
//    sums are read, and sent, as soon as they are there, while the tile before is
//    worked on, so that the other CTA's arrive before they are asked for.
// A row's maximum is raised, and its sums scaled down, only when it grows by more
// than 2^8.  All tiles of all (sequence, 128 rows) items are one line, cut evenly
// into one range per cluster; an item that spans ranges is left in parts in the
// workspace, which a second launch joins in the ranges' order.
//
// Precision: q and the cache enter exactly (an e4m3 cache as fp16 values, with q
// scaled by a power of two per row: 2^-38 of the row's largest).  Weights enter
// P V as bf16, 2^-8 of each (fp16 beside an e4m3 cache, 2^-11, or 2^-32 of the
// row's largest): independent errors, that stay below the result's own rounding
// to bf16 in the sum, while a second part would make the products 1.5 times as
// much where they bound the call.  Sums, statistics and parts are fp32.
//
// Every wait is bounded: one that gives up sets the device error word, after
// which the CTA's roles run through without waiting.
//
// Vectors that some rows see and others do not would reach the others as 0 * NaN
// if they are not finite: a segment whose sums are not all finite runs again; then
// each value that is not finite becomes 0 before P V, and a row that sees such a
// vector (its score is not finite) becomes NaN.
#include <utility>

#include "kq_attn_kernel.cuh"
#include "kq_vec.cuh"

namespace kq {
namespace attn {
namespace {

constexpr int LROWS = 128;               // rows of an item
constexpr int LSTART = 4;                // tiles' time that an item costs besides its tiles
constexpr float kGrow = 8.0f;            // log2 units that a row's maximum may lag behind
constexpr int SW = 16;                   // softmax warps
constexpr int HC = TK / 2;               // a softmax thread's positions of a tile
constexpr int XCHG = 32 * HC * 4;        // bytes that a warp sends per tile
constexpr int MOST_STAGES = 6;

template <int C, bool F8>
struct LCfg {
  static constexpr int NLOAD = 3;                     // loader warps
  static constexpr int TH = (SW + NLOAD + 1) * 32;    // softmax warps, loaders, products
  static constexpr int HD = C / 2;                    // dims of a CTA's half
  static constexpr int NB = HD / 64;                  // lines of a position, without the rope part's
  static constexpr int LINES = TK * 128;              // 64 dims of a tile's positions
  static constexpr int STAGE = (NB + 1) * LINES;      // the last lines: the rope part, in the first CTA
  static constexpr int QROPE = LROWS * 128;
  static constexpr int OROW = HD * 4 + 16;            // bytes of a row of sums on its way out, in q's and the ring's place
  // e4m3: 16 positions as they are in the cache, and how many such pieces a loader warp has on their way
  static constexpr int RAWROW = HD + 64, RAWS = F8 ? 3 : 0, RAW = RAWS * 16 * RAWROW;
  // Shared memory: q's rope part, the ring, the exchange (by quarters of the rows), the raw pieces, the line's index.
  static constexpr int smem(int stages, int quarters, int B) {
    return QROPE + stages * STAGE + 4 * quarters * XCHG + NLOAD * RAW + 4 * (B + 1);
  }
  static constexpr int ROOM = 227 * 1024 - 4096;  // less the static memory
  static_assert(smem(F8 ? 2 : 3, 4, 4096) <= ROOM, "all rows, the most sequences");
  static_assert(QROPE + (F8 ? 2 : 3) * STAGE + (F8 ? 4 * XCHG + NLOAD * RAW : 0) >= (F8 ? 32 : 128) * OROW, "and the sums on their way out");
  // tensor memory columns: q, S, P x 2, o
  static constexpr int CQ = 0, CS = HD / 2, CP = CS + TK, CO = CP + TK, COLS = 512;
  static constexpr float LIFT = F8 ? 7.0f : 0.0f;  // log2: fp16 weights, below 2^8, fill fp16's range
  static_assert(CO + HD <= COLS);
};

// A range's item that goes on in the next ranges.
struct Split {
  int b, rt, parts, slot;  // parts 0: none
};

struct LParams {
  AttnArgs a;  // one key-value head; G: heads
  const uint8_t* pool;
  int64_t page_bytes, slot_bytes;
  float c_scale;
  int rope, RT, clusters, rows;  // rows: of a part
  int stages, quarters;          // of the ring; of 32 rows that an item can have
  Split* split;
  float *part_ml, *part;
};

struct LBars {
  uint64_t full[MOST_STAGES], empty[MOST_STAGES], s_full[2], s_free, p_full[2], pv_done[2], q_full, x_full[SW], x_free[SW], decided[2][4];
  uint32_t tmem;
  int bad, peer_bad;
  int scan[NW];
  float back[LROWS];           // e4m3: the rows' powers of two
  float m[LROWS];              // the rows' maxima that their sums are relative to, in log2 units
  float top[4][LROWS];         // a warpgroup's half of a tile: the rows' largest score; at the end, its weight sums
};

// Shared-memory operand in 128-byte-swizzled groups of 8 lines (1024 bytes apart); mn_step: bytes from 64 values along M or
// N to the next (N-major operands).
__device__ __forceinline__ uint64_t line_desc(uint32_t saddr, uint32_t mn_step) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>((mn_step >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// kind::f16, fp32 accumulator, bf16 or fp16 operands, M = 128; n_major: B's N is contiguous
__device__ __forceinline__ constexpr uint32_t idesc(bool f16, int n, bool n_major) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
// Products issued by one lane of a converged warp (`on`), so that their operands can stay in uniform registers: moving
// them there for a lane's branch took twice the products' time.
__device__ __forceinline__ void mma_ts_on(uint32_t d_taddr, uint32_t a_taddr, uint64_t b_desc, uint32_t id, uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_taddr),
      "r"(a_taddr), "l"(b_desc), "r"(id), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ss_on(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc, uint32_t id, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.eq.u32 p, 0, 0;\n\tsetp.ne.u32 q, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_taddr),
      "l"(a_desc), "l"(b_desc), "r"(id), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_on(uint32_t bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }
// 16 bytes into the other CTA's shared memory; its barrier there counts them.
template <int TO>
__device__ __forceinline__ void send16(uint32_t dst, uint32_t bar, const float* x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0 + %6], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
               "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3])), "r"(bar), "n"(TO)
               : "memory");
}
__device__ __forceinline__ bool phase_done(uint64_t* bar, int phase) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(phase & 1)
               : "memory");
  return done != 0;
}
// After the wait for tensor-memory loads: uses of v stay behind it.
__device__ __forceinline__ void tie(uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
// The two warps of 32 rows that work on one tile.
__device__ __forceinline__ void rows_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(2 + id) : "memory"); }
// A copy of 16 bytes, both addresses with constant offsets.
template <int TO, int FROM>
__device__ __forceinline__ void copy16_at(uint32_t dst, const uint8_t* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0), "n"(TO), "n"(FROM) : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool finite16(uint32_t two, bool f16) {  // both halves
  const uint32_t e = f16 ? 0x7C00u : 0x7F80u;
  return (two & e) != e && (two >> 16 & e) != e;
}

template <int C, bool F8>
struct Latent {
  using L = LCfg<C, F8>;
  const LParams& p;
  const Seg g;
  LBars& bars;
  uint8_t* ring;
  uint8_t* qrope;
  uint8_t* xbuf;  // a softmax warp's place
  uint8_t* raw;   // a loader warp's
  uint32_t tb;    // tensor memory
  uint32_t rank;  // the CTA's half
  int tile0;      // tiles of earlier segments: the barriers' phases and the ring go on
  int xn;         // a softmax warp's tiles so far, as its exchange counts them
  bool ok;        // no wait has given up

  __device__ __forceinline__ void wait(uint64_t* bar, int phase) {
    if (!ok || __all_sync(0xFFFFFFFFu, phase_done(bar, phase))) return;
    bool done = false;
    for (uint32_t i = 0; i < kMaxPolls && !done; ++i) {
      done = mbar_try_wait(bar, static_cast<uint32_t>(phase & 1));
      done = __all_sync(0xFFFFFFFFu, done || phase_done(bar, phase));
    }
    ok = done && __all_sync(0xFFFFFFFFu, phase_done(bar, phase));
    if (!ok) record_error(p.a.err, DEV_ERR_MBAR_TIMEOUT);
  }

  // Both, which are mostly done already.
  __device__ __forceinline__ void wait(uint64_t* bar, int phase, uint64_t* bar2, int phase2) {
    if (!ok || __all_sync(0xFFFFFFFFu, phase_done(bar, phase) && phase_done(bar2, phase2))) return;
    wait(bar, phase);
    wait(bar2, phase2);
  }

  // Bytes from the pool's start to position j's vector; -1 where none is to be read.
  __device__ __forceinline__ int64_t offset_of(int j, int page) const {
    if (j < 0 || j >= g.len) return -1;
    if (page < 0 || page >= p.a.c.n_pages) {
      record_error(p.a.err, DEV_ERR_PAGE);
      return -1;
    }
    return page * p.page_bytes + (j & (p.a.c.page_size - 1)) * p.slot_bytes;
  }

  // ---- loaders: U positions at a time, in turn, their page ids one turn ahead
  __device__ __forceinline__ void load(int lw, int lane) {
    constexpr int NLOAD = L::NLOAD, U = F8 ? 16 : 32, PT = TK / U;
    const int n = g.t1 - g.t0, b0 = g.t0 * TK, units = PT * n;
    auto page_of = [&](int x) {  // of this lane's position
      const int j = b0 + U * x + lane % U;
      return x < units && j < g.len ? __ldg(g.table + (j >> p.a.page_shift)) : 0;
    };
    int page = page_of(lw);
    auto offset_at = [&](int x) {  // and its offset, the next page on its way
      const int next = page_of(x + NLOAD);
      const int64_t off = offset_of(b0 + U * x + lane % U, page);
      page = next;
      return off;
    };
    if constexpr (F8) {
      // Pieces come as they are, RAWS - 1 ahead, and go into their lines as fp16.
      constexpr int CH = L::HD / 16;  // 16-byte chunks of a row, without the rope part
      const int rch = p.rope / 16;    // 2 or 4
      auto fetch = [&](int x, int slot) {
        const int64_t off = x < units ? offset_at(x) : 0;
        const uint32_t to = smem_u32(raw) + slot * (16 * L::RAWROW);
        if (x < units && ok) {
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            const int r = (i * 32 + lane) / CH;
            const int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
            copy16(to + r * L::RAWROW + lane % CH * 16, p.pool + (src >= 0 ? src : 0) + rank * L::HD + lane % CH * 16, src >= 0);
          }
          for (int i = lane; i < 16 * rch; i += 32) {
            const int r = i / rch;
            const int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
            if (rank == 0) copy16(to + r * L::RAWROW + L::HD + i % rch * 16, p.pool + (src >= 0 ? src : 0) + C + i % rch * 16, src >= 0);
          }
        }
        copy_commit();
      };
#pragma unroll
      for (int i = 0; i < L::RAWS - 1; ++i) fetch(lw + i * NLOAD, i);
      int slot = 0;
      for (int x = lw; x < units; x += NLOAD) {
        const int gi = tile0 + x / PT, st = gi % p.stages;
        copy_wait<L::RAWS - 2>();
        __syncwarp();
        fetch(x + (L::RAWS - 1) * NLOAD, slot == 0 ? L::RAWS - 1 : slot - 1);
        if (gi >= p.stages) wait(&bars.empty[st], gi / p.stages - 1);
        uint8_t* lines = ring + st * L::STAGE + x % PT * (U * 128);
        const uint8_t* from = raw + slot * (16 * L::RAWROW);
        if (ok) {
#pragma unroll 4
          for (int i = 0; i < CH / 2; ++i) {
            const int r = (i * 32 + lane) / CH;
            put(lines + lane % CH / 4 * L::LINES, r, lane % CH % 4, *reinterpret_cast<const uint4*>(from + r * L::RAWROW + lane % CH * 16));
          }
          if (rank == 0)
            for (int i = lane; i < 16 * rch; i += 32)
              put(lines + L::NB * L::LINES, i / rch, i % rch, *reinterpret_cast<const uint4*>(from + i / rch * L::RAWROW + L::HD + i % rch * 16));
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars.full[st]);
        __syncwarp();  // the piece's place is free
        slot = slot + 1 == L::RAWS ? 0 : slot + 1;
      }
    } else {
      for (int x = lw; x < units; x += NLOAD) {
        const int gi = tile0 + x / PT, st = gi % p.stages;
        const int64_t off = offset_at(x);
        uint8_t* lines = ring + st * L::STAGE + x % PT * (U * 128);
        if (gi >= p.stages) wait(&bars.empty[st], gi / p.stages - 1);
        if (ok) {
          const bool rope = rank == 0 && (lane & 7) < p.rope / 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (lane >> 3) + 4 * i;
            int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
            const bool on = src >= 0;
            const uint8_t* from = p.pool + (on ? src : 0) + (lane & 7) * 16;
            const uint8_t* half = from + rank * (2 * L::HD);
            const uint32_t to = smem_u32(lines) + r * 128 + ((lane & 7) ^ (r & 7)) * 16;
            copy16_at<0, 0>(to, half, on);
            copy16_at<L::LINES, 128>(to, half, on);
            if constexpr (L::NB == 4) {
              copy16_at<2 * L::LINES, 256>(to, half, on);
              copy16_at<3 * L::LINES, 384>(to, half, on);
            }
            if (rope) copy16_at<L::NB * L::LINES, 2 * C>(to, from, on);
          }
        }
        // each thread's arrival, once its copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars.full[st])) : "memory");
      }
    }
    copy_commit();
    copy_wait<0>();
  }
  // 16 e4m3 values as fp16: chunks 2 c and 2 c + 1 of row r's line.
  static __device__ __forceinline__ void put(uint8_t* lines, int r, int c, uint4 v) {
    uint8_t* row = lines + r * 128;
    r &= 7;
    *reinterpret_cast<uint4*>(row + ((2 * c) ^ r) * 16) = make_uint4(f8_pair(v.x), f8_pair(v.x >> 16), f8_pair(v.y), f8_pair(v.y >> 16));
    *reinterpret_cast<uint4*>(row + ((2 * c + 1) ^ r) * 16) = make_uint4(f8_pair(v.z), f8_pair(v.z >> 16), f8_pair(v.w), f8_pair(v.w >> 16));
  }

  // ---- products, by one warp (its first lane issues): S of the next tile, P V of the oldest, whichever can run
  __device__ __forceinline__ void products(int lane, int segment) {
    const int n = g.t1 - g.t0;
    const uint32_t rs = smem_u32(ring), t = uniform(tb), on = elect();
    const uint64_t q = line_desc(smem_u32(qrope), 16);
    const int rope = rank == 0 ? p.rope / 16 : 0;
    wait(&bars.q_full, segment);
    uint32_t idle = 0;
    int sst = tile0 % p.stages, sph = tile0 / p.stages, vst = sst;  // the stages of both products' tiles
    for (int s = 0, v = 0; v < n && ok;) {
      bool did = false;
      const int gs = tile0 + s, gv = tile0 + v;
      if (s < n && __all_sync(0xFFFFFFFFu, phase_done(&bars.full[sst], sph) && (gs == 0 || phase_done(&bars.s_free, gs - 1)))) {
        fence_proxy_async_smem();  // the copies, which the barrier has put before this, seen by the tensor cores
        tc_fence_after();
        const uint64_t k = line_desc(uniform(rs + sst * L::STAGE), 16);
#pragma unroll
        for (int i = 0; i < L::HD / 16; ++i)
          mma_ts_on(t + L::CS, t + L::CQ + 8 * i, k + (i / 4 * L::LINES + i % 4 * 32) / 16, idesc(F8, TK, false), i > 0, on);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < rope) mma_ss_on(t + L::CS, q + i * 2, k + (L::NB * L::LINES + i * 32) / 16, idesc(F8, TK, false), on);
        commit_on(smem_u32(&bars.s_full[gs & 1]), on);
        ++s;
        if (++sst == p.stages) sst = 0, ++sph;
        did = true;
      }
      if (v < s && __all_sync(0xFFFFFFFFu, phase_done(&bars.p_full[gv & 1], gv >> 1))) {
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t c = line_desc(uniform(rs + vst * L::STAGE), L::LINES);
        const uint32_t w = uniform(t + L::CP + TK / 2 * (gv & 1));
#pragma unroll
        for (int k = 0; k < TK / 16; ++k) mma_ts_on(t + L::CO, w + 8 * k, c + k * 128, idesc(F8, L::HD, true), v > 0 || k > 0, on);
        commit_on(smem_u32(&bars.pv_done[gv & 1]), on);
        commit_on(smem_u32(&bars.empty[vst]), on);
        ++v;
        if (++vst == p.stages) vst = 0;
        did = true;
      }
      if (!did) __nanosleep(20);  // the slots are for the others
      idle = did ? 0 : idle + 1;
      if (idle > (1u << 25)) {
        ok = false;
        record_error(p.a.err, DEV_ERR_MBAR_TIMEOUT);
      }
    }
  }

  // ---- softmax: two threads per row and tile, half of its positions each; warps 0-7 take the even tiles, warps 8-15 the odd
  float l;
  bool poison;  // the row sees a vector that is not finite (careful run)

  // The row's half of q into tensor memory, its rope part into shared memory; mul: the row's power of two (e4m3 cache).
  __device__ __forceinline__ void load_q(const __nv_bfloat16* src, int r, uint32_t lanes, int part, bool active, float mul) {
    if (active) {
#pragma unroll
      for (int c = 0; c < L::HD / 8; c += 16) {
        const int col = part * (L::HD / 8) + c;
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = operand(src ? __ldg(reinterpret_cast<const uint4*>(src + rank * L::HD + 2 * col) + i) : make_uint4(0, 0, 0, 0), mul);
          v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        }
        tmem_st16(tb + lanes + L::CQ + col, v);
      }
      tmem_wait_st();
    }
    if (rank == 0)
      for (int c = part; c < p.rope / 8; c += 4)
        *reinterpret_cast<uint4*>(qrope + r * 128 + (c ^ (r & 7)) * 16) =
            operand(src && active ? __ldg(reinterpret_cast<const uint4*>(src + C) + c) : make_uint4(0, 0, 0, 0), mul);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.q_full);
  }
  static __device__ __forceinline__ uint4 operand(uint4 x, float mul) {
    if constexpr (F8) {
      auto two = [&](uint32_t v) {
        const float2 f = unpack2<false>(v);
        return pack2<true>(f.x * mul, f.y * mul);
      };
      return make_uint4(two(x.x), two(x.y), two(x.z), two(x.w));
    } else {
      return x;
    }
  }
  // Scales the row's sums in tensor memory, HD / 2 of them from column `sums` on, by c.
  static __device__ __forceinline__ void scale_sums(uint32_t sums, float c) {
#pragma unroll 1
    for (int d = 0; d < L::HD / 2; d += 16) {
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
  template <int... I>
  static __device__ __forceinline__ void send_all(uint32_t to, uint32_t bar, const float (&s)[HC], std::integer_sequence<int, I...>) {
    (send16<I * 512>(to, bar, s + 4 * I), ...);
  }
  // A tile's scores: this CTA's half of the sum from tensor memory, to the other CTA, and with the other's half added.  The
  // other CTA's warp has a place for one tile, which it says is free.
  __device__ __forceinline__ void exchange(float (&s)[HC], uint32_t lanes, int half) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t v[2][16];
#pragma unroll
    for (int c = 0; c < 2; ++c) tmem_ld16(tb + lanes + L::CS + HC * half + 16 * c, v[c]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      tie(v[c]);
#pragma unroll
      for (int e = 0; e < 16; ++e) s[16 * c + e] = __uint_as_float(v[c][e]);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars.s_free);
      mbar_arrive_expect_tx(&bars.x_full[warp], XCHG);
    }
    if (xn > 0) wait(&bars.x_free[warp], xn - 1);
    else __syncwarp();
    uint8_t* mine = xbuf + lane * 16;
    if (ok) {
      const uint32_t to = cluster_map(smem_u32(mine), rank ^ 1), bar = cluster_map(smem_u32(&bars.x_full[warp]), rank ^ 1);
      send_all(to, bar, s, std::make_integer_sequence<int, HC / 4>());
    }
    wait(&bars.x_full[warp], xn);
    ++xn;
#pragma unroll
    for (int c = 0; c < HC / 4; ++c) {
      const float4 x = *reinterpret_cast<const float4*>(mine + c * 512);
      const float2 lo = fadd2(make_float2(s[4 * c], s[4 * c + 1]), make_float2(x.x, x.y));
      const float2 hi = fadd2(make_float2(s[4 * c + 2], s[4 * c + 3]), make_float2(x.z, x.w));
      s[4 * c] = lo.x, s[4 * c + 1] = lo.y, s[4 * c + 2] = hi.x, s[4 * c + 3] = hi.y;
    }
    __syncwarp();
    if (lane == 0) arrive_remote(cluster_map(smem_u32(&bars.x_free[warp]), rank ^ 1));
  }
  // r: the row; f: from the raw product to log2 units.
  template <bool CAREFUL>
  __device__ __forceinline__ void softmax(uint32_t lanes, int r, bool active, int pos, uint64_t bits, float f) {
    const AttnArgs& a = p.a;
    const int n = g.t1 - g.t0, all_hi = g.len - a.T - 1, warp = threadIdx.x >> 5, wg = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const bool lead = (threadIdx.x & 31) == 0;
    float m = pos < 0 ? INFINITY : -INFINITY;  // padding: weights of 0 wherever masks are not looked at
    l = 0.0f;
    poison = false;
    for (int i = (tile0 & 1) ^ wg; i < n; i += 2) {
      const int gi = tile0 + i, tile = (g.t0 + i) * TK, base = tile + HC * half;
      float s[HC];
      float scale = f, mx = -INFINITY;
      wait(&bars.s_full[wg], gi >> 1);
      tc_fence_after();
      if (active) {
        exchange(s, lanes, half);
        if (!(f > 0.0f)) {  // a factor that turns the order around comes first
          scale = 1.0f;
#pragma unroll
          for (int e = 0; e < HC; ++e) s[e] *= f;
        }
        if (tile + TK - 1 > all_hi) {
#pragma unroll
          for (int e = 0; e < HC; ++e)
            if (!sees<true>(base + e, pos, bits, g.len - a.T, 0)) s[e] = -INFINITY;
        }
        if constexpr (CAREFUL) {
#pragma unroll
          for (int e = 0; e < HC; ++e)
            if (!finite(s[e])) {
              poison |= sees<true>(base + e, pos, bits, g.len - a.T, 0);
              s[e] = -INFINITY;
            }
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int e = 4; e < HC; e += 2) top[(e >> 1) & 3] = fmaxf(fmaxf(top[(e >> 1) & 3], s[e]), s[e + 1]);
        mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
      } else {
        tc_fence_before();
        __syncwarp();
        if (lead) mbar_arrive(&bars.s_free);
      }
      // P of two tiles ago is used up: its columns are free, and so is its barrier, at which a warp without rows must not
      // arrive for this tile before all others have for that one.  The tile before has its maxima; this one's are decided
      // after them.
      if (i > 1) wait(&bars.pv_done[wg], (gi - 2) >> 1, &bars.decided[wg ^ 1][quarter], (gi - 1) >> 1);
      else if (gi > 0) wait(&bars.decided[wg ^ 1][quarter], (gi - 1) >> 1);
      tc_fence_after();
      if (active) {
        const float now = bars.m[r];
        bars.top[2 * wg + half][r] = mx;
        rows_sync(wg * 4 + quarter);  // both halves know the maximum, old and new
        mx = fmaxf(mx, bars.top[2 * wg + (half ^ 1)][r]);
        if (now != m) {  // raised by the tile before
          l *= m == -INFINITY ? 0.0f : ex2(m - now);
          m = now;
        }
        const bool grow = mx > (m == -INFINITY ? m : m + kGrow);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float c = !grow ? 1.0f : m == -INFINITY ? 0.0f : ex2(m - mx);
          if (grow) {
            m = mx;
            if (half == 0) bars.m[r] = mx;
          }
          l *= c;
          if (i > 0) {
            wait(&bars.pv_done[wg ^ 1], (gi - 1) >> 1);
            tc_fence_after();
            scale_sums(tb + lanes + L::CO + half * (L::HD / 2), c);
            tc_fence_before();
          }
        }
      }
      __syncwarp();
      if (lead) mbar_arrive(&bars.decided[wg][quarter]);
      if (active) {
        const float mm = (m == -INFINITY ? 0.0f : m) - L::LIFT;  // nothing seen yet: the weights are 0
        const float2 sc = make_float2(scale, scale), off = make_float2(-mm, -mm);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < HC; e += 2) {
          const float2 x = ffma2(make_float2(s[e], s[e + 1]), sc, off);
          const float2 y = make_float2(ex2(x.x), ex2(x.y));
          sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], y);
          w[e / 2] = pack2<F8>(y.x, y.y);
        }
        tmem_st16(tb + lanes + L::CP + TK / 2 * wg + 16 * half, w);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
      }
      if constexpr (CAREFUL) {  // (static, as is all that is not inlined: an object with an address would live in memory)
        wait(&bars.full[gi % p.stages], gi / p.stages);
        clean(ring + gi % p.stages * L::STAGE + (warp & 7) * 1024);
      }
      tc_fence_before();
      __syncwarp();
      if (lead) mbar_arrive(&bars.p_full[wg]);
    }
    const int last = tile0 + n - 1;
    if (wg == (last & 1)) wait(&bars.pv_done[wg], last >> 1);
    softmax_sync();
    tc_fence_after();
    if (active) {  // relative to the rows' last maxima
      const float now = bars.m[r];
      if (now != m) l *= m == -INFINITY ? 0.0f : ex2(m - now);
    }
  }
  // Zeros in the place of a tile's values that are not finite, 8 positions per warp of the tile's eight: its scores are
  // done, its sums not begun.
  static __device__ __noinline__ void clean(uint8_t* lines) {
    const int lane = threadIdx.x & 31;
    for (int h = 0; h < L::NB; ++h) {
      uint32_t* x = reinterpret_cast<uint32_t*>(lines + h * L::LINES);
      for (int i = lane; i < 256; i += 32)
        if (!finite16(x[i], F8)) {
          const uint32_t e = F8 ? 0x7C00u : 0x7F80u;
          x[i] = ((x[i] & e) == e ? 0 : x[i] & 0xFFFFu) | ((x[i] >> 16 & e) == e ? 0 : x[i] & 0xFFFF0000u);
        }
    }
    fence_proxy_async_smem();
  }
};

template <int C, bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__((LCfg<C, F8>::TH), 1) latent_kernel(const __grid_constant__ LParams p) {
  using L = LCfg<C, F8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ LBars bars;
  const AttnArgs& a = p.a;
  uint8_t* qrope = smem;
  uint8_t* ring = qrope + L::QROPE;
  uint8_t* xbuf = ring + p.stages * L::STAGE;
  uint8_t* raw = xbuf + 4 * p.quarters * XCHG;
  int* prefix = reinterpret_cast<int*>(raw + L::NLOAD * L::RAW);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int range = blockIdx.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) { mbar_init(&bars.full[i], 32 * TK / (F8 ? 16 : 32)); mbar_init(&bars.empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 8);
      mbar_init(&bars.pv_done[i], 1);
      for (int w = 0; w < 4; ++w) mbar_init(&bars.decided[i][w], 2);
    }
    for (int w = 0; w < SW; ++w) { mbar_init(&bars.x_full[w], 1); mbar_init(&bars.x_free[w], 1); }
    mbar_init(&bars.s_free, 8);
    mbar_init(&bars.q_full, SW);
    fence_mbar_init();
  }
  if (warp == SW + L::NLOAD) { tmem_alloc(&bars.tmem, L::COLS); tmem_relinquish(); }
  pdl_wait();
  pdl_launch_dependents();
  build_prefix(a, LSTART, prefix, bars.scan);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tb = bars.tmem;
  const Line line(a, p.RT, prefix, p.clusters);
  const int lo = line.bound(min(range, line.nc)), hi = range < line.nc ? line.bound(range + 1) : lo;
  Split split = {0, 0, 0, 0};
  int tile0 = 0, segment = 0, xn = 0;
  bool ok = true;
  for (int u = lo; u < hi;) {
    const Item it(a, line, p.RT, LSTART, u);
    const int end = min(it.i1, hi);
    if (u < it.i0) u = it.i0;
    if (u >= end) {  // none of its tiles is in this range
      u = end;
      continue;
    }
    const int r0 = it.rt * LROWS, R = min(LROWS, a.T * a.G - r0);
    auto out_row = [&](int r) {
      return static_cast<__nv_bfloat16*>(a.out) + (static_cast<int64_t>(it.b) * a.T * a.G + r0 + r) * C + rank * L::HD;
    };
    if (it.len == 0) {
      for (int x = threadIdx.x; x < R * (L::HD / 4); x += L::TH) store4(out_row(x / (L::HD / 4)) + 4 * (x % (L::HD / 4)), make_float4(0, 0, 0, 0));
      u = end;
      continue;
    }
    Seg g;
    g.len = it.len;
    g.first = 0;
    g.table = a.page_table + it.b * a.max_pages;
    g.head_off = 0;
    g.t0 = u - it.i0;
    g.t1 = end - it.i0;
    const int r = threadIdx.x & (LROWS - 1), part = warp >> 2;  // softmax warps; part: of q's and the sums' dims
    const bool active = warp < SW && 32 * (warp & 3) < R;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int row = min(r0 + r, a.T * a.G - 1), t = row / a.G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(it.b) * a.T + t) * a.q_stride +
                             static_cast<int64_t>(row - t * a.G) * (C + p.rope);
    int pos = -1;
    uint64_t bits = 0;
    float f = a.scale * p.c_scale * 1.4426950408889634f, mul = 1.0f;
    if (warp < SW) {
      // a chain is a tree whose masks are known
      bits = tree_bits(a.tree ? __ldg(a.tree + static_cast<int64_t>(it.b) * a.T + t) : (2ull << t) - 1, a.T, t, g.len);
      pos = tree_position(bits, a.T, g.len);
    }
    if (warp < 4) bars.m[r] = pos < 0 ? INFINITY : -INFINITY;
    if (threadIdx.x == 0) bars.bad = bars.peer_bad = 0;
    if constexpr (F8) {
      if (warp < SW)  // the rows' largest values: a warp per row
        for (int r4 = warp * 4; r4 < R; r4 += 4 * SW) {
          uint4 v[4][3];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int x = min(r0 + r4 + k, a.T * a.G - 1), tt = x / a.G;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(it.b) * a.T + tt) * a.q_stride +
                                                              static_cast<int64_t>(x - tt * a.G) * (C + p.rope));
#pragma unroll
            for (int i = 0; i < 3; ++i) v[k][i] = lane + 32 * i < (C + p.rope) / 8 ? __ldg(src + lane + 32 * i) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < 3; ++i)
              for (uint32_t w : {v[k][i].x, v[k][i].y, v[k][i].z, v[k][i].w}) {
                const float2 y = unpack2<false>(w);
                mx = fmaxf(mx, fmaxf(fabsf(y.x), fabsf(y.y)));
              }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            // largest value into [2^13, 2^14); the factor and its inverse stay normal numbers
            const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 100);
            if (lane == 0) bars.back[r4 + k] = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
          }
        }
    }
    __syncthreads();  // the ring, the sums and tensor memory are free
    if constexpr (F8) {
      if (r < R) {
        f *= bars.back[r];
        mul = __uint_as_float((254u << 23) - __float_as_uint(bars.back[r]));  // its inverse
      }
    }
    Latent<C, F8> w{p, g, bars, ring, qrope, xbuf + ((warp >> 2) * p.quarters + (warp & 3)) * XCHG, raw + (warp - SW) * L::RAW, tb, rank, tile0, xn, ok, 0.0f, false};
    bool careful = false;
    for (;;) {
      if (warp < SW) {
        w.load_q(r < R ? q : nullptr, r, lanes, part, active, mul);
        if (!careful) {
          w.template softmax<false>(lanes, r, active, pos, bits, f);
          if (active) {
            bool bad = false;
#pragma unroll 1
            for (int d = part * (L::HD / 4); d < (part + 1) * (L::HD / 4); d += 16) {
              uint32_t v[16];
              tmem_ld16(tb + lanes + L::CO + d, v);
              tmem_wait_ld();
              tie(v);
#pragma unroll
              for (int i = 0; i < 16; ++i) bad |= !finite(__uint_as_float(v[i]));
            }
            if (bad && r < R) {
              bars.bad = 1;
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(smem_u32(&bars.peer_bad), rank ^ 1)), "r"(1) : "memory");
            }
          }
        } else {
          w.template softmax<true>(lanes, r, active, pos, bits, f);
        }
        bars.top[part][r] = pos < 0 ? 0.0f : w.poison ? NAN : w.l;  // padding: whatever the keys were
      } else if (warp < SW + L::NLOAD) {
        w.load(warp - SW, lane);
      } else {
        w.products(lane, segment);
      }
      ++segment;
      w.tile0 += g.t1 - g.t0;
      if (!w.ok)  // what is on its way to or from a CTA that did not wait for it lands before the CTA can end
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
      tc_fence_before();
      __syncwarp();
      cluster_sync();  // both CTAs have read what they were sent
      tc_fence_after();
      if (careful || !(bars.bad | bars.peer_bad)) break;
      careful = true;
      if (warp < 4) bars.m[r] = pos < 0 ? INFINITY : -INFINITY;
      cluster_sync();
    }
    tile0 = w.tile0;
    xn = w.xn;
    ok = w.ok;

    const bool whole = u == it.i0 && end == it.i1;
    const int slot = 2 * range + (lo >= it.i0 ? 1 : 0);  // the range starts in these tiles (1), or before them
    if (!whole && u == it.i0) split = {it.b, it.rt, line.range_of(it.i1 - 1) - range + 1, slot};
    // out through shared memory, in q's and the ring's place, a row of the half at a time
    if (active) {
      const float weight = (bars.top[0][r] + bars.top[1][r]) + (bars.top[2][r] + bars.top[3][r]);
      const float inv = weight == 0.0f ? 0.0f : p.c_scale / weight;
      uint8_t* stage = smem + r * L::OROW;
#pragma unroll 1
      for (int d = part * (L::HD / 4); d < (part + 1) * (L::HD / 4); d += 16) {
        uint32_t v[16];
        tmem_ld16(tb + lanes + L::CO + d, v);
        tmem_wait_ld();
        tie(v);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          float4 x = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
          if (pos < 0) x = make_float4(0, 0, 0, 0);
          if (whole) put4(reinterpret_cast<__nv_bfloat16*>(stage) + d + i, x, inv);
          else *reinterpret_cast<float4*>(stage + (d + i) * 4) = x;
        }
      }
      if (!whole && part == 0 && rank == 0 && r < R)
        *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(slot) * p.rows + r) * 2) = make_float2(pos < 0 ? -INFINITY : bars.m[r], weight);
      fence_proxy_async_smem();
    }
    if (warp < SW) {
      softmax_sync();
      if (part == 0 && r < R) {
        void* dst = whole ? static_cast<void*>(out_row(r)) : p.part + (static_cast<int64_t>(slot) * p.rows + r) * C + rank * L::HD;
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(smem + r * L::OROW)),
                     "r"(whole ? L::HD * 2 : L::HD * 4)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
      }
    }
    tc_fence_before();
    __syncthreads();  // the copies have read the ring; weights and maxima are read before the next segment writes them
    tc_fence_after();
    u = end;
  }
  if (threadIdx.x == 0 && rank == 0) p.split[range] = split;
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == SW + L::NLOAD) tmem_dealloc(tb, L::COLS);
}

// Joins the parts of the items that span ranges: o = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k, in the ranges' order.
// A block: a range's item, eight rows of it (a warp each) or, with MANY parts expected, one row, its parts in eight shares.
constexpr int JTH = 256;
template <int C, bool MANY>
__global__ void __launch_bounds__(JTH) latent_join_kernel(const __grid_constant__ LParams p) {
  constexpr int V = C / 128, JW = JTH / 32, MOST = 160;  // vectors of a row per lane; ranges
  __shared__ float factor[MANY ? 1 : JW][MOST];
  __shared__ float4 sums[MANY ? JW : 1][C / 4];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 s4 = __ldcg(reinterpret_cast<const int4*>(p.split) + blockIdx.x);
  const Split sp = {s4.x, s4.y, s4.z, s4.w};
  const int r = MANY ? blockIdx.y : blockIdx.y * JW + warp;
  const int64_t row0 = static_cast<int64_t>(sp.rt) * LROWS;
  if (sp.parts == 0 || row0 + (MANY ? r : r - warp) >= p.a.T * p.a.G) return;
  const bool on = row0 + r < p.a.T * p.a.G;
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
  if (on) {
#pragma unroll 4
    for (int k = MANY ? warp : 0; k < sp.parts; k += MANY ? JW : 1) {
      const float4* part = reinterpret_cast<const float4*>(p.part + (static_cast<int64_t>(slot_of(k)) * p.rows + r) * C) + lane;
#pragma unroll
      for (int i = 0; i < V; ++i) add4(acc[i], e[k], __ldcg(part + 32 * i));
    }
  }
  const float inv = ll == 0.0f ? 0.0f : p.c_scale / ll;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + (static_cast<int64_t>(sp.b) * p.a.T * p.a.G + row0 + r) * C;
  if (!MANY) {
    if (on)
#pragma unroll
      for (int i = 0; i < V; ++i) put4(out + 4 * (lane + 32 * i), acc[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) sums[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    if (threadIdx.x < C / 4) {
      float4 x = sums[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < JW; ++k) add4(x, 1.0f, sums[k][threadIdx.x]);
      put4(out + 4 * threadIdx.x, x, inv);
    }
  }
}

int clusters() { return num_sms() / 2 < 160 ? num_sms() / 2 : 160; }

struct LLayout {
  int rows;
  size_t ml_off, part_off, bytes;
};
LLayout latent_layout(int C, int64_t T, int H) {
  LLayout l;
  l.rows = static_cast<int>(min_i64(LROWS, T * H));
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t slots = 2 * static_cast<size_t>(clusters());
  l.ml_off = up(clusters() * sizeof(Split));
  l.part_off = l.ml_off + up(slots * l.rows * 2 * sizeof(float));
  l.bytes = l.part_off + up(slots * l.rows * C * sizeof(float));
  return l;
}

template <int C, bool F8>
cudaError_t launch_halves(LParams p, cudaStream_t st) {
  using L = LCfg<C, F8>;
  p.quarters = (p.rows + 31) / 32;
  p.stages = F8 ? 2 : 3;  // and as many more as there is room for
  while (p.stages < MOST_STAGES && L::smem(p.stages + 1, p.quarters, p.a.B) <= L::ROOM) ++p.stages;
  const size_t smem = L::smem(p.stages, p.quarters, p.a.B);
  static int set[64] = {0};
  const int dev = current_device_id();
  if (set[dev] < static_cast<int>(smem)) {
    const cudaError_t e = cudaFuncSetAttribute(latent_kernel<C, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    set[dev] = static_cast<int>(smem);
  }
  cudaError_t e = launch_pdl(latent_kernel<C, F8>, dim3(2 * p.clusters), dim3(L::TH), smem, st, p);
  if (e != cudaSuccess) return e;
  // few items: many parts of each
  const bool many = static_cast<int64_t>(p.a.B) * p.RT * 8 <= p.clusters;
  if (many) return launch_pdl(latent_join_kernel<C, true>, dim3(p.clusters, p.rows), dim3(JTH), 0, st, p);
  return launch_pdl(latent_join_kernel<C, false>, dim3(p.clusters, (p.rows + 7) / 8), dim3(JTH), 0, st, p);
}

}  // namespace
}  // namespace attn

size_t latent_workspace_bytes(const kq_latent_cache& l, int64_t T, int H) {
  return attn::latent_layout(l.latent_dim, T < 1 ? 1 : T, H).bytes;
}

cudaError_t launch_latent(const LatentArgs& x, cudaStream_t st) {
  attn::LParams p = {};
  p.a.c.dtype = x.l.dtype;
  p.a.c.n_kv_heads = 1;
  p.a.c.page_size = x.l.page_size;
  p.a.c.n_pages = x.l.n_pages;
  p.a.page_table = x.page_table;
  p.a.max_pages = x.max_pages;
  p.a.seq_lens = x.seq_lens;
  p.a.q = x.q;
  p.a.q_stride = x.q_stride;
  p.a.out = x.out;
  p.a.scale = x.scale;
  p.a.B = x.B;
  p.a.T = x.T;
  p.a.Hq = p.a.G = x.H;
  p.a.page_shift = x.page_shift;
  p.a.room = x.room;
  p.a.err = x.err;
  p.a.tree = x.tree;
  const int es = x.l.dtype == KQ_BF16 ? 2 : 1;
  p.pool = static_cast<const uint8_t*>(x.l.c);
  p.page_bytes = x.l.page_stride * es;
  p.slot_bytes = x.l.slot_stride * es;
  p.c_scale = x.l.scale;
  p.rope = x.l.rope_dim;
  p.RT = (x.T * x.H + attn::LROWS - 1) / attn::LROWS;
  p.clusters = attn::clusters();
  const attn::LLayout l = attn::latent_layout(x.l.latent_dim, x.T, x.H);
  p.rows = l.rows;
  uint8_t* ws = static_cast<uint8_t*>(x.ws);
  p.split = reinterpret_cast<attn::Split*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + l.ml_off);
  p.part = reinterpret_cast<float*>(ws + l.part_off);
  if (x.l.latent_dim == 512) return x.l.dtype == KQ_BF16 ? attn::launch_halves<512, false>(p, st) : attn::launch_halves<512, true>(p, st);
  return x.l.dtype == KQ_BF16 ? attn::launch_halves<256, false>(p, st) : attn::launch_halves<256, true>(p, st);
}

}  // namespace kq
