// kq_latent.cu -- attention of the newest T tokens of each sequence over its
// cache of latent vectors c_j, which all heads share, in absorbed form:
//   s_j = scale q.c_j (latent and rope part),  o = sum_j softmax(s)_j c_j[0 .. C)
// in one pass with a running maximum and running sums, on the 5th-generation
// tensor cores.
//
// Bound: a vector of 1152 bytes (C = 512, bf16) serves 2 (2 C + 64) flops per row
// (a token's head): up to 64 rows the bytes bound it, with 128 rows 242 flops per
// byte stand against the device's 282.  What is in the way is the room.  128 rows'
// sums, 512 fp32 values each, would be all of an SM's tensor memory and their
// queries 144 KB of its shared memory; so a CTA, one per SM, takes up to 64 rows.
// Its products:
//   S   = Q K^T    rows are the M (128 lanes, the upper ones idle), 32 positions the N;
//                  Q in tensor memory (64 rows: three of its nine lines of 64 dims in
//                  shared memory), K lines in shared memory
//   O^T += V^T P^T dims are the M, 128 at a time, the rows the N: 16, 32 or 64 columns
//                  of sums per 128 dims.  V^T is the same lines, M-major; P rows lie in
//                  shared memory as K-major lines, so nothing is transposed
// With rows as O's M all calls would pay for 128 of them.
//
// (Two CTAs that share 128 rows by halves of the dims load and multiply nothing
// twice, but have to exchange the scores' halves: 32 KB per 64 positions through
// the cluster's shared memory took 2000 clocks by itself, the tile 6300: 64
// sequences of 4096 positions and 128 heads 171 us, and 99 us with 16 heads.)
//
// Warps:
//  * loaders copy 16 positions at a time into a ring of stages of 32, 64 dims of
//    a position a line of 128 bytes in the matrix descriptors' 128-byte swizzle
//    (e4m3: 8 positions, as they are, into places of their own, and from there as
//    fp16, exactly, into the lines);
//  * two warps issue the products, S of the next tiles and O of the oldest;
//  * softmax warps, two threads per row and tile, half of its positions each; two
//    groups of them take every other tile, as a tile's chain of steps is longer
//    than its share of the time.  A row's maximum is raised only when it grows by
//    more than 2^24 (e4m3 cache: 2^11);
//  * four warps then scale the sums down, before this tile's are added.
// All tiles of all (sequence, rows) items are one line, cut evenly into one range
// per CTA (row tiles of a sequence side by side where that leaves no SM over: a
// line of sequences, which neighbouring CTAs walk together); an item that spans
// ranges is left in parts in the workspace, which a second launch joins in the
// ranges' order.  The loaders do not wait for a segment's end: the next one's first
// tiles are there when its queries are (64 sequences of 4096 positions, 128 heads
// 145 -> 140 us, e4m3, 16 heads, 96 -> 90).
//
// Precision: q and the cache enter exactly (an e4m3 cache as fp16 values, with q
// scaled by a power of two per row: 2^-38 of the row's largest).  Weights enter
// the second product as bf16, 2^-8 of each (fp16 beside an e4m3 cache, 2^-11, or
// 2^-29 of the row's largest), and the rounded weights are the ones that are
// summed: with p_j (1 + e_j) in both sums the result is off by
// sum_j p_j e_j (c_j - o).  That is next to nothing for a row that one position
// dominates (as the maximum may lag, its weight is any number, not 1: summed before
// the rounding, it had an error of the whole row), and where many count, the e_j are
// independent.  A second part of the weights would be half as many products again
// where they bound the call.  Sums, statistics and parts are fp32.
//
// Measured on one GB300, calls in a graph: 64 sequences of 4096 positions, 16
// heads, bf16, 69 us (4.4 TB/s; a tile is 1600 clocks, at the memory's rate, but the
// first one comes 18000 clocks after the start); 128 heads 140 us (520 TFLOP/s; a
// tile is 1800 clocks: of a stage's 8700 from one load to the next, 4000 pass until
// its copies are there and 4500 until its sums are done, and five stages are all that
// fits); in an e4m3 cache 90 and 198 us (four or three stages beside the raw pieces);
// one of 131071 positions, 16 heads, 47 us, of which the join takes 10; one of 1000,
// 15 us.
//
// Every wait is bounded: one that gives up sets the device error word, after
// which the CTA's roles run through without waiting.
//
// Vectors that some rows see and others do not would reach the others as 0 * NaN
// if they are not finite: segments whose sums are not all finite run again once the
// range is through; then each value that is not finite becomes 0 before the second
// product, and a row that sees such a vector (its score is not finite) becomes NaN.
#include "kq_attn_kernel.cuh"
#include "kq_join.cuh"
#include "kq_vec.cuh"

namespace kq {
namespace attn {
namespace {

constexpr int LT = 32;                // positions per tile
constexpr int HC = LT / 2;            // a softmax thread's positions of a tile
// Tiles' time that an item costs besides its tiles: its queries and first vectors come, its sums go.  (32 sequences of up to
// 16001 positions, 128 heads: 121 us; counted as 4, 150.)
constexpr int LSTART = 20;
constexpr int MOST_ROWS = 64, MOST_STAGES = 8;
// Warps 0-15 by four: the first two of each four are softmax warps (their tensor memory lanes are rows 0-31 and 32-63), of
// the others one each issues the two products, and six load; warps 16-19 scale sums.  (One warp that issued whichever
// product could run saw both late: 64 sequences of 4096 positions, 128 heads, 165 us in place of 153.)
constexpr int LTH = 20 * 32, SCORES = 2, SUMS = 3, NLOAD = 6;

template <int C, bool F8, int NR>
struct LCfg {
  static constexpr int NB = C / 64 + 1;               // lines of a position, the rope part's last
  static constexpr int LINES = LT * 128;              // 64 dims of a tile's positions
  static constexpr int STAGE = NB * LINES;
  static constexpr int QT = C == 512 && NR == 64 ? 6 : NB;  // lines of q in tensor memory
  static constexpr int QS = (NB - QT) * NR * 128;     // the others, in shared memory
  static constexpr int P = NR * 128;                  // a tile's weights
  static constexpr int U = F8 ? 8 : 16;               // positions at a time of a loader
  // e4m3: the places of a loader's pieces, as they are in the cache; all but one are on their way
  static constexpr int RAWROW = C + 64, RAWS = F8 ? 2 : 0, RAW = RAWS * U * RAWROW;
  static constexpr int smem(int stages, int B) { return QS + 2 * P + stages * STAGE + NLOAD * RAW + 4 * (B + 1); }
  static constexpr int ROOM = 227 * 1024 - 4096;      // less the static memory
  static constexpr int LEAST = F8 ? 3 : 4;            // stages
  static_assert(smem(LEAST, kMaxSeqs) <= ROOM);
  // tensor memory columns: o, q, S x 2
  static constexpr int MB = C / 128, CO = 0, CQ = C == 256 ? 256 : NR == 64 ? 256 : 128, CS = 448, COLS = 512;
  static_assert(MB * NR <= CQ && CQ + 32 * QT <= CS && CS + 2 * LT <= COLS);
  // log2 units that a row's maximum may lag behind, so that sums are seldom scaled (a scaling takes a
  // tile's time, and of 64 rows one grows by 8 units in every fourth tile): bf16 weights have fp32's range; fp16 ones, which end
  // at 2^16, are lifted so far that what is left below reaches 2^-28 of the maximum
  static constexpr float GROW = F8 ? 11.0f : 24.0f, LIFT = F8 ? 4.0f : 0.0f;
};

struct LParams {
  AttnArgs a;  // one key-value head; G: heads
  const uint8_t* pool;
  int64_t page_bytes, slot_bytes;
  float c_scale;
  int rope, RT, rows, ranges, stages;  // rows: of a part
  int abreast;                         // row tiles of a sequence that go side by side: RT, or 1
  int by_item;                         // split [items] instead of [ranges]
  Split* split;
  float *part_ml, *part;
};

constexpr int FLAGS = 32;
struct LBars {
  uint64_t full[MOST_STAGES], empty[MOST_STAGES], s_full[2], s_free[2], p_full[2], pv_done[2], q_full, decided[2][2], grown[2], scaled[2];
  uint32_t tmem;
  int bad;                       // a segment's sums are not all finite; which segments of the range's (the last: and all behind it)
  uint32_t flags[FLAGS];
  int scan[NW];
  int raise[2];                  // a warpgroup's last tile, counted from 1, that raised a maximum
  float m[MOST_ROWS];            // the rows' maxima that their sums are relative to, in log2 units
  float factor[2][MOST_ROWS];    // a warpgroup's tile: what the sums are scaled by; at the end [0]: the rows' last factor
  float top[4][MOST_ROWS];       // a warpgroup's half of a tile: the rows' largest score; at the end, weight sums (e4m3, before: q's largest values)
  float weight[MOST_ROWS];
  int seen[MOST_ROWS];           // 0: padding
};

// Shared-memory operand in 128-byte-swizzled groups of 8 lines (1024 bytes apart); mn_step: bytes from 64 values along M or
// N to the next (operands whose M or N is contiguous).
__device__ __forceinline__ uint64_t line_desc(uint32_t saddr, uint32_t mn_step) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>((mn_step >> 4) & 0x3FFF) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// kind::f16, fp32 accumulator, bf16 or fp16 operands, M = 128; m_major: A's M is contiguous
__device__ __forceinline__ constexpr uint32_t idesc(bool f16, int n, bool m_major) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (m_major ? 1u << 15 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
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
__device__ __forceinline__ void mma_ss_on(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc, uint32_t id, uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_taddr),
      "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate), "r"(on)
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
__device__ __forceinline__ bool phase_done(uint64_t* bar, int phase) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(done)
               : "r"(smem_u32(bar)), "r"(phase & 1)
               : "memory");
  return done != 0;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
// After the wait for tensor-memory loads: uses of v stay behind it.
template <int N>
__device__ __forceinline__ void tie(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// All but the loaders, which run ahead.
__device__ __forceinline__ void others_sync() { asm volatile("bar.sync 6, %0;" ::"n"(LTH - 32 * NLOAD) : "memory"); }
// The two warps of 32 rows that work on one tile.
__device__ __forceinline__ void rows_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(2 + id) : "memory"); }
// A copy of 16 bytes, both addresses with constant offsets.
template <int TO, int FROM>
__device__ __forceinline__ void copy16_at(uint32_t dst, const uint8_t* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0), "n"(TO), "n"(FROM) : "memory");
}
__device__ __forceinline__ bool finite16(uint32_t two, bool f16) {  // both halves
  const uint32_t e = f16 ? 0x7C00u : 0x7F80u;
  return (two & e) != e && (two >> 16 & e) != e;
}

__device__ __forceinline__ float largest(uint32_t two) {  // of two bf16 values, by size
  const float2 y = unpack2<false>(two);
  return fmaxf(fabsf(y.x), fabsf(y.y));
}

template <int C, bool F8, int NR>
struct Latent {
  using L = LCfg<C, F8, NR>;
  const LParams& p;
  const Seg g;
  LBars& bars;
  uint8_t *qs, *ps, *ring, *raw;
  uint32_t tb;  // tensor memory
  int tile0;    // tiles of earlier segments: the barriers' phases and the ring go on
  bool ok;      // no wait has given up

  __device__ __forceinline__ void wait(uint64_t* bar, int phase) {
    if (!ok || __all_sync(0xFFFFFFFFu, phase_done(bar, phase))) return;
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar, static_cast<uint32_t>(phase & 1), p.a.err));
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
    constexpr int U = L::U, PT = LT / U, STEP = NLOAD;
    static_assert(STEP <= 3 * PT && L::LEAST >= 3);
    // A loader's turns go on from segment to segment, at most three tiles apart: one that stood out a few short segments could
    // come to a barrier two phases early, and take the phase before the last for the last.
    const int first = (lw + STEP - tile0 % STEP * PT % STEP) % STEP;
    const int n = g.t1 - g.t0, b0 = g.t0 * LT, units = PT * n;
    auto page_of = [&](int x) {  // of this lane's position
      const int j = b0 + U * x + lane % U;
      return x < units && j < g.len ? __ldg(g.table + (j >> p.a.page_shift)) : 0;
    };
    int page = page_of(first);
    auto offset_at = [&](int x) {  // and its offset, the next page on its way
      const int next = page_of(x + STEP);
      const int64_t off = offset_of(b0 + U * x + lane % U, page);
      page = next;
      return off;
    };
    if constexpr (F8) {
      constexpr int CH = C / 16;    // 16-byte chunks of a row, without the rope part
      const int rch = p.rope / 16;  // 2 or 4
      auto fetch = [&](int x, int slot) {
        const int64_t off = x < units ? offset_at(x) : 0;
        const uint32_t to = smem_u32(raw) + slot * (U * L::RAWROW);
        if (x < units && ok) {
#pragma unroll
          for (int i = 0; i < U * CH / 32; ++i) {
            const int r = (i * 32 + lane) / CH;
            const int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
            copy16(to + r * L::RAWROW + lane % CH * 16, p.pool + (src >= 0 ? src : 0) + lane % CH * 16, src >= 0);
          }
          const int r = lane / rch & (U - 1);
          const int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
          if (lane < U * rch) copy16(to + r * L::RAWROW + C + lane % rch * 16, p.pool + (src >= 0 ? src : 0) + C + lane % rch * 16, src >= 0);
        }
        copy_commit();
      };
#pragma unroll
      for (int i = 0; i < L::RAWS - 1; ++i) fetch(first + i * STEP, i);
      int slot = 0;
      for (int x = first; x < units; x += STEP) {
        const int gi = tile0 + x / PT, st = gi % p.stages;
        copy_wait<L::RAWS - 2>();
        __syncwarp();
        fetch(x + (L::RAWS - 1) * STEP, slot == 0 ? L::RAWS - 1 : slot - 1);
        if (gi >= p.stages) wait(&bars.empty[st], gi / p.stages - 1);
        uint8_t* lines = ring + st * L::STAGE + x % PT * (U * 128);
        const uint8_t* from = raw + slot * (U * L::RAWROW);
        if (ok) {
#pragma unroll 4
          for (int i = 0; i < U * CH / 32; ++i) {
            const int r = (i * 32 + lane) / CH;
            put(lines + lane % CH / 4 * L::LINES, r, lane % CH % 4, *reinterpret_cast<const uint4*>(from + r * L::RAWROW + lane % CH * 16));
          }
          if (lane < U * rch)
            put(lines + (L::NB - 1) * L::LINES, lane / rch, lane % rch, *reinterpret_cast<const uint4*>(from + lane / rch * L::RAWROW + C + lane % rch * 16));
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars.full[st]);
        __syncwarp();  // the piece's place is free
        slot = slot + 1 == L::RAWS ? 0 : slot + 1;
      }
    } else {
      for (int x = first; x < units; x += STEP) {
        const int gi = tile0 + x / PT, st = gi % p.stages;
        const int64_t off = offset_at(x);
        uint8_t* lines = ring + st * L::STAGE + x % PT * (U * 128);
        if (gi >= p.stages) wait(&bars.empty[st], gi / p.stages - 1);
        if (ok) {
          const bool rope = (lane & 7) < p.rope / 8;
#pragma unroll
          for (int i = 0; i < U / 4; ++i) {
            const int r = (lane >> 3) + 4 * i;
            const int64_t src = __shfl_sync(0xFFFFFFFFu, off, r);
            const bool on = src >= 0;
            const uint8_t* from = p.pool + (on ? src : 0) + (lane & 7) * 16;
            const uint32_t to = smem_u32(lines) + r * 128 + ((lane & 7) ^ (r & 7)) * 16;
            copy16_at<0, 0>(to, from, on);
            copy16_at<L::LINES, 128>(to, from, on);
            copy16_at<2 * L::LINES, 256>(to, from, on);
            copy16_at<3 * L::LINES, 384>(to, from, on);
            if constexpr (C == 512) {
              copy16_at<4 * L::LINES, 512>(to, from, on);
              copy16_at<5 * L::LINES, 640>(to, from, on);
              copy16_at<6 * L::LINES, 768>(to, from, on);
              copy16_at<7 * L::LINES, 896>(to, from, on);
            }
            if (rope) copy16_at<(L::NB - 1) * L::LINES, 2 * C>(to, from, on);
          }
        }
        // each thread's arrival, once its copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars.full[st])) : "memory");
      }
    }
    if constexpr (F8) copy_wait<0>();
  }
  // 16 e4m3 values as fp16: chunks 2 c and 2 c + 1 of row r's line.
  static __device__ __forceinline__ void put(uint8_t* lines, int r, int c, uint4 v) {
    uint8_t* row = lines + r * 128;
    r &= 7;
    *reinterpret_cast<uint4*>(row + ((2 * c) ^ r) * 16) = make_uint4(f8_pair(v.x), f8_pair(v.x >> 16), f8_pair(v.y), f8_pair(v.y >> 16));
    *reinterpret_cast<uint4*>(row + ((2 * c + 1) ^ r) * 16) = make_uint4(f8_pair(v.z), f8_pair(v.z >> 16), f8_pair(v.w), f8_pair(v.w >> 16));
  }

  // ---- products, each by a warp of its own
  __device__ __forceinline__ void scores(int segment) {
    const int n = g.t1 - g.t0;
    const uint32_t rs = smem_u32(ring), t = uniform(tb), on = elect();
    const uint64_t q = line_desc(smem_u32(qs), 16);
    const int rope = p.rope / 16;
    wait(&bars.q_full, segment);
    int st = tile0 % p.stages, ph = tile0 / p.stages;
    for (int i = 0; i < n; ++i) {
      const int gi = tile0 + i;
      wait(&bars.full[st], ph);
      if (gi > 1) wait(&bars.s_free[gi & 1], (gi - 2) >> 1);
      fence_proxy_async_smem();  // the copies, which the barrier has put before this, seen by the tensor cores
      tc_fence_after();
      if (ok) {
        const uint64_t k = line_desc(uniform(rs + st * L::STAGE), 16);
        const uint32_t to = uniform(t + L::CS + LT * (gi & 1));
#pragma unroll
        for (int j = 0; j < 4 * L::NB; ++j) {
          if (j >= 4 * (L::NB - 1) && j - 4 * (L::NB - 1) >= rope) continue;
          const uint64_t b = k + (j / 4 * L::LINES + j % 4 * 32) / 16;
          if (j < 4 * L::QT) mma_ts_on(to, t + L::CQ + 8 * j, b, idesc(F8, LT, false), j > 0, on);
          else mma_ss_on(to, q + ((j / 4 - L::QT) * (NR * 128) + j % 4 * 32) / 16, b, idesc(F8, LT, false), 1, on);
        }
        commit_on(smem_u32(&bars.s_full[gi & 1]), on);
      }
      if (++st == p.stages) st = 0, ++ph;
    }
  }
  __device__ __forceinline__ void sums() {
    const int n = g.t1 - g.t0;
    const uint32_t rs = smem_u32(ring), t = uniform(tb), on = elect();
    const uint64_t w0 = line_desc(smem_u32(ps), 16);
    int st = tile0 % p.stages;
    for (int i = 0; i < n; ++i) {
      const int gi = tile0 + i;
      wait(&bars.scaled[gi & 1], gi >> 1);
      wait(&bars.p_full[gi & 1], gi >> 1);
      tc_fence_after();
      if (ok) {
        const uint64_t c = line_desc(uniform(rs + st * L::STAGE), L::LINES);
        const uint64_t w = w0 + uniform((gi & 1) * L::P / 16);
        const uint32_t more = i > 0;
#pragma unroll
        for (int k = 0; k < LT / 16; ++k)
#pragma unroll
          for (int mb = 0; mb < L::MB; ++mb)
            mma_ss_on(t + L::CO + mb * NR, c + (2 * mb * L::LINES + k * 2048) / 16, w + 2 * k, idesc(F8, NR, true), k > 0 ? 1 : more, on);
        commit_on(smem_u32(&bars.pv_done[gi & 1]), on);
        commit_on(smem_u32(&bars.empty[st]), on);
      }
      if (++st == p.stages) st = 0;
    }
  }

  // ---- softmax: two threads per row and tile, half of its positions each; the first warpgroup takes the even tiles
  float l;
  bool poison;  // the row sees a vector that is not finite (careful run)

  // Part `part` of four of the row's q; mul: the row's power of two (e4m3 cache).
  __device__ __forceinline__ void load_q(const __nv_bfloat16* src, int r, uint32_t lanes, int part, bool active, float mul) {
    const int W = C + p.rope;
    auto chunk = [&](int d) {  // 8 dims from d on
      return operand(src && d < W ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0, 0, 0, 0), mul);
    };
    if (active) {
#pragma unroll
      for (int c = 0; c < (2 * L::QT + 3) / 4; ++c) {
        const int col = 16 * (part + 4 * c);
        if (col < 32 * L::QT) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = chunk(2 * col + 8 * i);
            v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
          }
          tmem_st16(tb + lanes + L::CQ + col, v);
        }
      }
      tmem_wait_st();
      if (r < NR)
        for (int c = part; c < 8 * (L::NB - L::QT); c += 4)
          *reinterpret_cast<uint4*>(qs + c / 8 * (NR * 128) + r * 128 + ((c & 7) ^ (r & 7)) * 16) = chunk(64 * L::QT + 8 * c);
    }
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
      const int gi = tile0 + i, tile = (g.t0 + i) * LT, base = tile + HC * half;
      float s[HC];
      float scale = f, mx = -INFINITY;
      wait(&bars.s_full[wg], gi >> 1);
      tc_fence_after();
      if (active) {
        {
          uint32_t v[HC];
          tmem_ld16(tb + lanes + L::CS + LT * wg + HC * half, v);
          tmem_wait_ld();
          tie(v);
#pragma unroll
          for (int e = 0; e < HC; ++e) s[e] = __uint_as_float(v[e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lead) mbar_arrive(&bars.s_free[wg]);
        if (!(f > 0.0f)) {  // a factor that turns the order around comes first
          scale = 1.0f;
#pragma unroll
          for (int e = 0; e < HC; ++e) s[e] *= f;
        }
        if (tile + LT - 1 > all_hi) {
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
        if (lead) mbar_arrive(&bars.s_free[wg]);
      }
      // P of two tiles ago is used up: its place is free, and so are its barriers, at which a warp without rows must not
      // arrive for this tile before all others have for that one.  The tile before has its maxima; this one's are decided
      // after them.
      if (i > 1) wait(&bars.pv_done[wg], (gi - 2) >> 1, &bars.decided[wg ^ 1][quarter], (gi - 1) >> 1);
      else if (gi > 0) wait(&bars.decided[wg ^ 1][quarter], (gi - 1) >> 1);
      if (active) {
        const float now = bars.m[r];
        bars.top[2 * wg + half][r] = mx;
        rows_sync(wg * 2 + quarter);  // both halves know the maximum, old and new
        mx = fmaxf(mx, bars.top[2 * wg + (half ^ 1)][r]);
        if (now != m) {  // raised by the tile before
          l *= m == -INFINITY ? 0.0f : ex2(m - now);
          m = now;
        }
        const bool grow = mx > (m == -INFINITY ? m : m + L::GROW);
        float c = 1.0f;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          if (grow) {
            c = m == -INFINITY ? 0.0f : ex2(m - mx);
            m = mx;
            l *= c;
            if (half == 0) bars.m[r] = mx;
            bars.raise[wg] = gi + 1;
          }
        }
        if (half == 0 && r < NR) bars.factor[wg][r] = c;
      }
      __syncwarp();
      if (lead) {
        mbar_arrive(&bars.decided[wg][quarter]);
        mbar_arrive(&bars.grown[wg]);
      }
      if (active) {
        const float mm = (m == -INFINITY ? 0.0f : m) - L::LIFT;  // nothing seen yet: the weights are 0
        const float2 sc = make_float2(scale, scale), off = make_float2(-mm, -mm);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        uint32_t w[HC / 2];
#pragma unroll
        for (int e = 0; e < HC; e += 2) {
          const float2 x = ffma2(make_float2(s[e], s[e + 1]), sc, off);
          w[e / 2] = pack2<F8>(ex2(x.x), ex2(x.y));
          sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], unpack2<F8>(w[e / 2]));  // of the weights as they are multiplied
        }
        if (r < NR) {
          uint8_t* line = ps + wg * L::P + r * 128;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<uint4*>(line + ((2 * half + c) ^ (r & 7)) * 16) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        fence_proxy_async_smem();
      }
      if constexpr (CAREFUL) {  // (static, as is all that is not inlined: an object with an address would live in memory)
        wait(&bars.full[gi % p.stages], gi / p.stages);
        clean(ring + gi % p.stages * L::STAGE, 2 * half + quarter);
      }
      __syncwarp();
      if (lead) mbar_arrive(&bars.p_full[wg]);
    }
    const int last = tile0 + n - 1;
    if (wg == (last & 1)) wait(&bars.pv_done[wg], last >> 1);
    softmax_sync();
    if (active) {  // relative to the rows' last maxima
      const float now = bars.m[r];
      if (now != m) l *= m == -INFINITY ? 0.0f : ex2(m - now);
    }
    // the rows' weight sums, and what their sums are multiplied by (padding: nothing, whatever the keys were)
    bars.top[2 * wg + half][r] = pos < 0 ? 0.0f : poison ? NAN : l;
    softmax_sync();
    if (wg == 0 && half == 0) {
      const float weight = (bars.top[0][r] + bars.top[1][r]) + (bars.top[2][r] + bars.top[3][r]);
      bars.weight[r] = weight;
      bars.factor[0][r] = weight == 0.0f ? 0.0f : p.c_scale / weight;
    }
  }
  // Zeros in the place of a tile's values that are not finite, 8 positions per warp of the tile's four: its scores are done,
  // its sums not begun.
  static __device__ __noinline__ void clean(uint8_t* stage, int quarter) {
    const int lane = threadIdx.x & 31;
    for (int h = 0; h < L::NB - 1; ++h) {
      uint32_t* x = reinterpret_cast<uint32_t*>(stage + h * L::LINES + quarter * (L::LINES / 4));
      for (int i = lane; i < L::LINES / 16; i += 32)
        if (!finite16(x[i], F8)) {
          const uint32_t e = F8 ? 0x7C00u : 0x7F80u;
          x[i] = ((x[i] & e) == e ? 0 : x[i] & 0xFFFFu) | ((x[i] >> 16 & e) == e ? 0 : x[i] & 0xFFFF0000u);
        }
    }
    fence_proxy_async_smem();
  }

  // ---- the sums, of 32 of each 128 dims per warp: scaled when a tile has raised a row's maximum, before its own are added
  __device__ __forceinline__ void rescale(uint32_t lanes) {
    const int n = g.t1 - g.t0;
    for (int i = 0; i < n; ++i) {
      const int gi = tile0 + i, wg = gi & 1;
      wait(&bars.grown[wg], gi >> 1);
      if (i > 0 && bars.raise[wg] == gi + 1) {
        wait(&bars.pv_done[wg ^ 1], (gi - 1) >> 1);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < L::MB * NR; c += 16) {
          uint32_t v[16];
          tmem_ld16(tb + lanes + L::CO + c, v);
          tmem_wait_ld();
          tie(v);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * bars.factor[wg][(c & (NR - 1)) + e]);
          tmem_st16(tb + lanes + L::CO + c, v);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bars.scaled[wg]);
    }
  }
};

template <int C, bool F8, int NR>
__global__ void __launch_bounds__(LTH, 1) latent_kernel(const __grid_constant__ LParams p) {
  using L = LCfg<C, F8, NR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ LBars bars;
  const AttnArgs& a = p.a;
  uint8_t* ps = smem + L::QS;
  uint8_t* ring = ps + 2 * L::P;
  uint8_t* raw = ring + p.stages * L::STAGE;
  int* prefix = reinterpret_cast<int*>(raw + NLOAD * L::RAW);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool softmax = warp < 16 && (warp & 3) < 2, scaler = warp >= 16;
  const int loader = !softmax && !scaler && warp > 3 ? (warp >> 2) * 2 + (warp & 3) - 4 : -1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) { mbar_init(&bars.full[i], 32 * LT / L::U); mbar_init(&bars.empty[i], 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_free[i], 4);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.pv_done[i], 1);
      mbar_init(&bars.decided[i][0], 2);
      mbar_init(&bars.decided[i][1], 2);
      mbar_init(&bars.grown[i], 4);
      mbar_init(&bars.scaled[i], 4);
      bars.raise[i] = 0;
    }
    bars.bad = 0;
    for (int i = 0; i < FLAGS; ++i) bars.flags[i] = 0;
    mbar_init(&bars.q_full, 8);
    fence_mbar_init();
  }
  if (warp == SCORES) { tmem_alloc(&bars.tmem, L::COLS); tmem_relinquish(); }
  pdl_wait();
  pdl_launch_dependents();
  build_prefix<LT>(a, LSTART, prefix, bars.scan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = bars.tmem, lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  // row tiles abreast: neighbouring CTAs take the same range of a line of sequences, each for its row tile, and the ranges
  // of one row tile are numbered in a row
  const int most = gridDim.x / p.abreast, at = blockIdx.x / p.abreast, side = blockIdx.x - at * p.abreast, RT = p.RT / p.abreast;
  const Line line(a, RT, prefix, most);
  const int range = side * most + at, lo = line.bound(min(at, line.nc)), hi = at < line.nc ? line.bound(at + 1) : lo;
  auto note = [&](const Item& it, bool whole, int slot) {
    const int item = (it.b * line.HR + it.hr) * p.abreast + side;
    if (!whole) p.split[p.by_item ? item : range] = {item, range, line.range_of(it.i1 - 1) - at + 1, slot};
    else if (p.by_item) p.split[item].parts = 0;
  };
  if (threadIdx.x == 0 && !p.by_item) p.split[range].parts = 0;
  int tile0 = 0, segment = 0, pass = 0, u = lo, number = 0;  // segment: that ran; number: in this pass
  bool ok = true;
  for (;;) {
    if (u >= hi) {  // the segments whose sums are not all finite run again
      if (pass++ > 0) break;
      __syncthreads();
      if (!bars.bad) break;
      u = lo;
      number = 0;
      continue;
    }
    const Item it(a, line, RT, LSTART, u);
    const int end = min(it.i1, hi);
    if (u < it.i0) u = it.i0;
    if (u >= end) {  // none of its tiles is in this range
      u = end;
      continue;
    }
    const int r0 = (it.rt + side) * NR, R = min(NR, a.T * a.G - r0);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (static_cast<int64_t>(it.b) * a.T * a.G + r0) * C;
    if (it.len == 0) {
      if (threadIdx.x == 0) note(it, true, 0);
      if (scaler)
        for (int x = threadIdx.x - 512; x < R * (C / 4); x += LTH - 512) store4(out + 4 * x, make_float4(0, 0, 0, 0));
      u = end;
      continue;
    }
    const int name = min(number++, 32 * FLAGS - 1);
    if (pass > 0 && !(bars.flags[name >> 5] >> (name & 31) & 1)) {
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
    const int r = 32 * (warp & 3) + lane, part = warp >> 2;  // softmax warps: the row, and which of four parts of the work
    const bool active = softmax && 32 * (warp & 3) < R;
    const int row = min(r0 + r, a.T * a.G - 1), t = row / a.G;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(it.b) * a.T + t) * a.q_stride +
                             static_cast<int64_t>(row - t * a.G) * (C + p.rope);
    int pos = -1;
    uint64_t bits = 0;
    float f = a.scale * p.c_scale * 1.4426950408889634f, mul = 1.0f;
    if (softmax) {
      // a chain is a tree whose masks are known
      bits = tree_bits(a.tree ? __ldg(a.tree + static_cast<int64_t>(it.b) * a.T + t) : (2ull << t) - 1, a.T, t, g.len);
      pos = tree_position(bits, a.T, g.len);
      if (part == 0) {
        bars.m[r] = pos < 0 ? INFINITY : -INFINITY;
        bars.seen[r] = r < R && pos >= 0;
      }
    }
    if constexpr (F8) {
      if (softmax) {  // the row's largest value into [2^13, 2^14); the factor and its inverse stay normal numbers
        float mx = 0.0f;
        if (r < R)
#pragma unroll 6
          for (int c = part; c < (C + p.rope) / 8; c += 4) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(q) + c);
            mx = fmaxf(mx, fmaxf(fmaxf(largest(x.x), largest(x.y)), fmaxf(largest(x.z), largest(x.w))));
          }
        bars.top[part][r] = mx;
        softmax_sync();
        mx = fmaxf(fmaxf(bars.top[0][r], bars.top[1][r]), fmaxf(bars.top[2][r], bars.top[3][r]));
        const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 127);
        f *= __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
        mul = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
      }
    }
    Latent<C, F8, NR> w{p, g, bars, smem, ps, ring, raw + max(loader, 0) * L::RAW, tb, tile0, ok, 0.0f, false};
    const bool whole = u == it.i0 && end == it.i1;
    const int slot = 2 * range + (lo >= it.i0 ? 1 : 0);  // the range starts in these tiles (1), or before them
    if (u == it.i0 && threadIdx.x == 0) note(it, whole, slot);
    if (loader >= 0) {  // on to the next segment as soon as there is room
      w.load(loader, lane);
      w.tile0 += g.t1 - g.t0;
    } else {
      if (softmax) {
        softmax_sync();  // the rows' maxima are there
        w.load_q(r < R ? q : nullptr, r, lanes, part, active, mul);
        if (pass == 0) w.template softmax<false>(lanes, r, active, pos, bits, f);
        else w.template softmax<true>(lanes, r, active, pos, bits, f);
      } else if (scaler) {
        w.rescale(lanes);
      } else if (warp == SCORES) {
        w.scores(segment);
      } else {
        w.sums();
      }
      ++segment;
      w.tile0 += g.t1 - g.t0;
      others_sync();  // the sums are complete, and the rows' factors there
      tc_fence_after();
      if (warp != 16 && warp != 17) {
        // a warp's lanes are 32 of each 128 dims; loaders are not there, so of the upper ones two warps each take half of the
        // columns, of the lower ones the softmax warps a quarter
        const int of = (warp & 2) ? 2 : 4, span = NR * L::MB / of, col0 = ((warp & 2) ? warp >> 4 : part) * span;
        bool bad = false;
#pragma unroll 1
        for (int c = col0; c < col0 + span; c += 8) {
          const int c0 = c % NR, d = c / NR * 128 + r;
          if (c0 >= R) continue;
          float* to = p.part + static_cast<int64_t>(slot) * p.rows * C + d;
          uint32_t v[8];
          tmem_ld8(tb + lanes + L::CO + c, v);
          tmem_wait_ld();
          tie(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int rr = c0 + e;
            if (rr < R) {
              const float x = bars.seen[rr] ? __uint_as_float(v[e]) : 0.0f;
              bad |= !finite(x);
              if (whole) out[rr * C + d] = __float2bfloat16_rn(x * bars.factor[0][rr]);
              else to[rr * C] = x;
            }
          }
          __syncwarp();
        }
        if (bad && pass == 0) {
          bars.bad = 1;
          atomicOr(&bars.flags[name >> 5], 1u << (name & 31));
        }
      }
      if (scaler && !whole && threadIdx.x - 512 < R) {
        const int rr = threadIdx.x - 512;
        *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(slot) * p.rows + rr) * 2) =
            make_float2(bars.seen[rr] ? bars.m[rr] : -INFINITY, bars.weight[rr]);
      }
      tc_fence_before();
      others_sync();  // what lies in shared and tensor memory is read
      tc_fence_after();
    }
    tile0 = w.tile0;
    ok = w.ok;
    u = end;
  }
  copy_commit();
  copy_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == SCORES) tmem_dealloc(tb, L::COLS);
}

int ranges() { return num_sms() < 160 ? num_sms() : 160; }
// Rows of an item: 16, 32 or 64 columns of sums.
int rows_of(int64_t all) { return all <= 16 ? 16 : all <= 32 ? 32 : MOST_ROWS; }

struct LLayout {
  int rows;
  size_t ml_off, part_off, bytes;
};
LLayout latent_layout(int C, int64_t T, int H) {
  LLayout l;
  l.rows = rows_of(T * H);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t slots = 2 * static_cast<size_t>(ranges());
  l.ml_off = up(ranges() * sizeof(Split));
  l.part_off = l.ml_off + up(slots * l.rows * 2 * sizeof(float));
  l.bytes = l.part_off + up(slots * l.rows * C * sizeof(float));
  return l;
}

template <int C, bool F8, int NR>
cudaError_t launch_rows(LParams p, cudaStream_t st) {
  using L = LCfg<C, F8, NR>;
  p.stages = L::LEAST;  // and as many more as there is room for
  while (p.stages < MOST_STAGES && L::smem(p.stages + 1, p.a.B) <= L::ROOM) ++p.stages;
  const size_t smem = L::smem(p.stages, p.a.B);
  static bool set[64] = {false};
  const int dev = current_device_id();
  if (!set[dev]) {  // for all calls: one at the same time may want less
    const cudaError_t e = cudaFuncSetAttribute(latent_kernel<C, F8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ROOM);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const cudaError_t e = launch_pdl(latent_kernel<C, F8, NR>, dim3(p.ranges), dim3(LTH), smem, st, p);
  if (e != cudaSuccess) return e;
  return launch_join<C, __nv_bfloat16>(JoinParams{p.a, p.split, p.part_ml, p.part, p.RT, p.rows, p.by_item, p.c_scale}, p.ranges, st);
}
template <int C, bool F8>
cudaError_t launch_type(const LParams& p, cudaStream_t st) {
  return p.rows == 16 ? launch_rows<C, F8, 16>(p, st) : p.rows == 32 ? launch_rows<C, F8, 32>(p, st) : launch_rows<C, F8, MOST_ROWS>(p, st);
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
  const attn::LLayout l = attn::latent_layout(x.l.latent_dim, x.T, x.H);
  p.rows = l.rows;
  p.RT = (x.T * x.H + p.rows - 1) / p.rows;
  p.ranges = attn::ranges();
  // Row tiles side by side read the same vectors at the same time, so the second one finds them in L2, but only where next to
  // no SM is left over by it.  us, side by side / one after the other, bf16:
  //   no SM over    2 row tiles: 1000 positions 22.6/22.9, 131071 70.9/73.1, 64 x 4096 141/147, 256 x 500 138/141
  //                 4: 16 x 8192 124.5/129.3   8: 8 x 8192 123.8/126.7   19: 4 x 8192 142.2/142.4
  //   2 SMs over    3: 16 x 8192 100.4/102.5   5: 8 x 8192 86.7/88.7   6: 99.3/101.4   10: 150.6/153.0   15: 118.6/119.9
  //   more          7 (5 over): 113.5/113.6    9 (8): 141.4/139.7      16 (8): 235.5/228.8
  // and beside an e4m3 cache, where the conversion is what takes time, within 1% of each other up to 2 SMs over.
  p.abreast = p.ranges % p.RT <= 2 ? p.RT : 1;
  p.ranges -= p.ranges % p.abreast;
  p.by_item = static_cast<int64_t>(x.B) * p.RT <= p.ranges;
  uint8_t* ws = static_cast<uint8_t*>(x.ws);
  p.split = reinterpret_cast<attn::Split*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + l.ml_off);
  p.part = reinterpret_cast<float*>(ws + l.part_off);
  if (x.l.latent_dim == 512) return x.l.dtype == KQ_BF16 ? attn::launch_type<512, false>(p, st) : attn::launch_type<512, true>(p, st);
  return x.l.dtype == KQ_BF16 ? attn::launch_type<256, false>(p, st) : attn::launch_type<256, true>(p, st);
}

}  // namespace kq
