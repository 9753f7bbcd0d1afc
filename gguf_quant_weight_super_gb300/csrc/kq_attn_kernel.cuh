// kq_attn_kernel.cuh -- attention of the newest T tokens of each sequence over
// its paged cache (instantiated per cache and query type in
// kq_attn_<cache>_<query>.cu, launched by kq_attn.cu):
//   s_j = scale q.k_j  or  softcap tanh(scale q.k_j / softcap)
//   o   = sum_j 2^(s_j log2 e - m) v_j / sum_j 2^(s_j log2 e - m)
// over the positions j that the token sees, in one pass with a running
// maximum m and running sums (the sums are scaled down when m grows).
//
// Bound: the cache is read once and every key and value serves the T*G query
// rows of its head only, so up to about 64 rows the bytes bound it.  Hence
//  * the rows of a head (T tokens x G heads) share what is loaded.  They are
//    the N of the matrix instructions, 8 to 32 per pass over the cache, and
//    positions (scores) and values' dims (sums) the M: S^T = K q^T, then
//    o^T += V^T w^T.  With rows as M, 16 of them would be the least, while
//    most decode steps have 8 or fewer; the weights go from one product's
//    result to the next one's operand by 8 x 8 transposes between lanes;
//  * each warp streams its own sub-tiles of 16 positions through its own ring
//    of asynchronous 16-byte copies (any page size, order of slots and
//    alignment of lengths: a row is one token of one head) and keeps its own
//    m and sums, so no barrier interrupts the loads; the four warps' sums
//    join once per segment.  Rows are padded by 16 bytes in shared memory, so
//    that the 8-row matrix loads touch every bank once;
//  * all tiles of 64 positions of all (sequence, head, row tile) items are one
//    line, cut evenly into one contiguous range per CTA, whatever the
//    lengths (each item counts three tiles more than it has, what starting and
//    ending it costs: a batch of 24 ragged sequences, among them one of a
//    single position, took 115 us without).  An item inside one range is finished there; for one that spans
//    ranges the CTAs leave their sums in the workspace, and the last to
//    arrive joins them in the ranges' order (so the result does not depend on
//    which one that is).
//
// Precision: products enter the matrix instructions exactly or in parts.
// bf16 cache: bf16 q as it is, fp32 q as three bf16 parts (all 24 bits); the
// weights 2^(..) as two parts (2^-17) for bf16 q and three for fp32 q.  e4m3
// cache: its values are fp16 values, so fp16 instructions serve; q is scaled
// by a power of two per row into fp16's range (bf16: one part; fp32: two, 22
// bits), weights are two parts of 2^15 times their value (the sums of weights
// likewise), which are exact to 2^-22 of a weight or to 2^-40 of the row's
// largest one: fp16 ends at 2^-24, and the many small weights beside a peak
// would vanish without the factor.  Accumulation is fp32; the matrix instructions
// cut what they add to an accumulator instead of rounding it, which over the
// hundreds of steps of a long range grows to 2^-16, so with fp32 q each step's
// product is added by rounding fp32 additions.
//
// Measured on one GB300, calls in a graph: 4 x 131071 positions, 32 heads on 8
// of 128, bf16, 308-322 us (6.4-6.6 TB/s, 94-98% of the copy rate); 24 sequences
// of 0 to 9001 positions, 72.5 us (5.4 TB/s: the median SM has read its ranges
// after 54 us, the slowest fifth, the same SMs each time, after 60 to 62, and an
// even cut cannot know them; the joins end at 69); one of 1000 positions, 9.4 us,
// a chain of length, page, row, sum, partial sums and their join; 16 sequences in
// an e4m3 cache, heads of 256, fp32 q, window 4096, cap, 34 us (3.9 TB/s: two CTAs
// per SM of 255 registers, and 4 us of joins).
//
// Values that no row sees are never loaded (zeros take their place).  One that
// some rows of the block see and others do not would reach the others as
// 0 * NaN if it is not finite: a warp whose sums are not all finite runs its
// part again, taking those values out of the product and adding each to the
// rows that see it.
//
// TREE: the newest tokens are a tree, whose masks say what a row sees of them;
// tiles that end before them are as above.  Parts then stay in the workspace for
// a second launch (kq_join.cuh), since a tree's rows are many and one SM's time to
// join them showed: 16 nodes of 4 heads a group over 1000 positions, 8 heads of
// 128, 15 us in place of 30.  4 x 24 nodes, window 4096, e4m3, heads of 256, fp32
// q: 43 us.
#pragma once

#include "kq_cache.h"

namespace kq {
namespace attn {

// What a first launch leaves of an item to a second one (kq_join.cuh): (sequence * heads + head) * RT + row tile, the first
// range, the parts (0: none), the first one's place.  The other ranges' lie at 2 * range + 1.
struct Split {
  int item, range, parts, slot;
};

struct Params;
// The second launch of a tree's call (kq_attn.cu): rows of an item's part, heads of D values, fp32 or bf16 out.
cudaError_t launch_tree_join(const Params& p, int rows, int D, bool f32, int ranges, cudaStream_t st);

constexpr int NW = 4;            // warps per CTA
constexpr int NTH = NW * 32;
constexpr int WT = 16;           // positions per warp sub-tile
constexpr int TK = NW * WT;      // positions per tile
constexpr int START = 3;         // tiles' time that an item costs besides its tiles

// The attention kernel's static shared memory.
struct Scratch {
  int scan[NW], last;
};
// Trees: what each query row of a pass sees of the drafted tokens, and its position (-1: padding).
template <int ROWS>
struct TreeRows {
  uint64_t bits[ROWS];
  int pos[ROWS];
};

template <class Q, class C, int D, int NT>
struct Cfg {
  static constexpr bool F8 = sizeof(C) == 1, QF32 = sizeof(Q) == 4;
  static constexpr int ROWS = 8 * NT;
  static constexpr int NQ = F8 ? (QF32 ? 2 : 1) : (QF32 ? 3 : 1);  // parts of q
  static constexpr int NP = F8 ? 2 : (QF32 ? 3 : 2);               // parts of the weights
  static constexpr float LIFT = 32768.0f;                          // of fp16 weights, which reach 65504
  static constexpr int RB = D * static_cast<int>(sizeof(C)) + 16;  // bytes of a cache row in shared memory
  static constexpr int SUB = WT * RB, STAGE = 2 * SUB;
  static constexpr int QB = 2 * D + 16;  // bytes of a q row in shared memory
  static constexpr int QBYTES = NQ * ROWS * QB;
  static constexpr int HDR = (ROWS * (2 + 2 * NW) * 4 + 127) / 128 * 128;  // row scales, the join's and the warps' statistics
  static constexpr int FIXED = HDR + QBYTES;
  // CTAs per SM: three where the sums take few registers, two where a ring of at least two stages fits beside q in half of
  // the shared memory, else one.  An SM has 228 KB, of which each CTA's static memory and 1 KB of the system's go off; what
  // the budgets leave is the line of tiles' index, 4 bytes per sequence (large batches have fewer CTAs per SM).
  static constexpr int budget(int ctas) { return (ctas == 3 ? 73 : ctas == 2 ? 110 : 192) * 1024; }
  static constexpr int stages(int ctas) { return (budget(ctas) - FIXED) / (NW * STAGE); }
  static constexpr int CPS = NT * D <= 128 && stages(3) >= 2 ? 3 : stages(2) >= 2 ? 2 : 1;
  static constexpr int S = stages(CPS) < 6 ? stages(CPS) : 6;  // ring stages
  static constexpr int RING = S * NW * STAGE, SMEM = FIXED + RING;
  static_assert(CPS * (SMEM + 4 * 257 + static_cast<int>(sizeof(Scratch) + sizeof(TreeRows<ROWS>)) + 1024) <= 228 * 1024, "256 sequences: all resident");
  static constexpr bool QREG = NT * NQ * (D / 8) <= 32;  // q's operands stay in registers
  static constexpr int OB = (D + 4) * 4;                 // bytes of a row of the warps' sums in shared memory
  static_assert(S >= 2 && S * STAGE >= ROWS * OB, "the warps' sums take the ring's place");
};

struct Params {
  AttnArgs a;
  int RT;          // row tiles per (sequence, head)
  float* part;     // [2 * grid][ROWS][D] sums, then [2 * grid][ROWS][2] maximum and weight sum
  float* part_ml;
  int* count;      // [grid] arrivals at the split item whose first tile a range holds
  Split* split;    // trees: [items] or, if those are more than ranges, [grid]
  int by_item;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// An 8 x 8 tile of 16-bit values held as matrix operands are (row lane / 4, columns 2 (lane & 3) and + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two values as packed 16-bit ones (lo in the low half), and back.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// e4m3 values of the low two bytes as two fp16 (exact).
__device__ __forceinline__ uint32_t f8_pair(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void put4(float* p, float4 v, float f) {
  *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 v, float f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2<false>(v.x * f, v.y * f), pack2<false>(v.z * f, v.w * f));
}
__device__ __forceinline__ void add4(float4& a, float f, float4 v) {
  a = make_float4(fmaf(f, v.x, a.x), fmaf(f, v.y, a.y), fmaf(f, v.z, a.z), fmaf(f, v.w, a.w));
}
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// ---- trees of drafted tokens

// What token t of a tree sees of the drafted tokens, and its position (-1: padding).  With a window the tokens behind it are
// taken out: padding, which stands at -1 wherever a bit names it, and tokens too far up the tree.  Whole warps call: which
// tokens are padding their lanes find together, in the time of the token's own mask (each token's masks by itself: 4 x 24
// nodes, window 4096, 0.6 us of 43).
struct TreeToken {
  uint64_t bits;
  int pos;
  __device__ __forceinline__ TreeToken(const AttnArgs& a, int b, int t, int len) {
    const uint64_t* masks = a.tree + static_cast<int64_t>(b) * a.T;
    auto bits_of = [&](int u) { return tree_bits(__ldg(masks + u), a.T, u, len); };
    uint64_t token = ~0ull;  // those that are no padding
    if (a.window > 0) {
      const int lane = threadIdx.x & 31;
      const uint32_t lower = __ballot_sync(0xFFFFFFFFu, lane < a.T && bits_of(min(lane, a.T - 1)) != 0);
      const uint32_t upper = __ballot_sync(0xFFFFFFFFu, lane + 32 < a.T && bits_of(min(lane + 32, a.T - 1)) != 0);
      token = static_cast<uint64_t>(upper) << 32 | lower;
    }
    bits = bits_of(t);
    pos = tree_position(bits, a.T, len);
    if (a.window > 0 && pos - a.window >= -1) {
      const int n = __popcll(bits);
      bits &= token;
      if (n > a.window)  // (as many tokens as the window has can stand after the context)
        for (uint64_t rest = bits; rest != 0; rest &= rest - 1) {
          const int u = __ffsll(static_cast<long long>(rest)) - 1;
          if (tree_position(bits_of(u), a.T, len) <= pos - a.window) bits &= ~(1ull << u);
        }
    }
  }
};

// Whether a token (its position pos; bits: of a tree) sees the slot of position j, base being the first new token's.
template <bool TREE>
__device__ __forceinline__ bool sees(int j, int pos, uint64_t bits, int base, int window) {
  if constexpr (TREE) {
    const int u = j - base;
    if (u >= 0) return u < 64 && (bits >> u & 1);
  }
  return j <= pos && (window == 0 || j > pos - window);
}

// One segment: tiles [t0, t1) of one item, for one warp.
struct Seg {
  const int32_t* table;  // the sequence's pages
  int64_t head_off;      // elements
  int len, first;        // positions [first, len) can be seen by some row
  int t0, t1;
};

// What a warp keeps of a tree: the rows' bits, in shared memory, and the position of the first new token's slot.  (Nothing in
// a chain's warps, whose values the careful run holds in memory.)
template <bool TREE>
struct WarpTree {
  const uint64_t* tree;
  int first_new;
};
template <>
struct WarpTree<false> {};

template <class Q, class C, int D, int NT, bool TREE>
struct Warp : WarpTree<TREE> {
  using K = Cfg<Q, C, D, NT>;
  // o[n][d]: dims 16 d + ... (M) of rows 8 n + ... (N): registers 0, 1 of the lane's first dim, 2, 3 of its second, for rows
  // 8 n + 2 (lane & 3) and + 1
  float o[NT][D / 16][4];
  float m[NT][2], l[NT][2];  // those rows' maximum (in log2 units) and this lane's part of the weight sum

  // The copies of one sub-tile: K rows, then V rows.  `page`: this lane's row's page id (row lane & 15).
  static __device__ __forceinline__ void issue(const Params& p, const Seg& g, uint32_t stage, int base, int page, int lane) {
    const AttnArgs& a = p.a;
    constexpr int CH = D * static_cast<int>(sizeof(C)) / 16;  // 16-byte chunks per row
    if (base >= g.first && base + WT <= g.len && a.c.page_size >= WT / 2 &&
        __all_sync(0xFFFFFFFFu, static_cast<unsigned>(page) < a.c.n_pages)) {
      // two times eight whole rows of one page, at one stride
      const int64_t row = a.c.slot_stride * static_cast<int64_t>(sizeof(C));
      uint32_t dst = stage + lane / CH * K::RB + lane % CH * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int pg = __shfl_sync(0xFFFFFFFFu, page, 8 * h);
        int64_t src = (pg * a.c.page_stride + g.head_off) * static_cast<int64_t>(sizeof(C)) +
                      (((base + 8 * h) & (a.c.page_size - 1)) + lane / CH) * row + lane % CH * 16;
#pragma unroll
        for (int i = 0; i < CH / 4; ++i) {
          copy16(dst, static_cast<const uint8_t*>(a.c.k) + src, true);
          copy16(dst + K::SUB, static_cast<const uint8_t*>(a.c.v) + src, true);
          src += 32 / CH * row;
          dst += 32 / CH * K::RB;
        }
      }
    } else {
      issue_rows(p, g, stage, base, page, lane);
    }
  }
  static __device__ __noinline__ void issue_rows(const Params& p, const Seg& g, uint32_t stage, int base, int page, int lane) {
    const AttnArgs& a = p.a;
    constexpr int CH = D * static_cast<int>(sizeof(C)) / 16;
    const int j = base + (lane & 15);
    bool on = j >= g.first && j < g.len;
    if (on && (page < 0 || page >= a.c.n_pages)) {
      record_error(a.err, DEV_ERR_PAGE);
      on = false;
    }
    const int64_t off = on ? (page * a.c.page_stride + (j & (a.c.page_size - 1)) * a.c.slot_stride + g.head_off) *
                                 static_cast<int64_t>(sizeof(C))
                           : -1;
#pragma unroll 1
    for (int i = 0; i < CH / 2; ++i) {
      const int c = i * 32 + lane, row = c / CH, col = c % CH;
      const int64_t ro = __shfl_sync(0xFFFFFFFFu, off, row);
      const bool ok = ro >= 0;
      const int64_t src = (ok ? ro : 0) + col * 16;
      const uint32_t dst = stage + row * K::RB + col * 16;
      copy16(dst, static_cast<const uint8_t*>(a.c.k) + src, ok);
      copy16(dst + K::SUB, static_cast<const uint8_t*>(a.c.v) + src, ok);
    }
  }
  static __device__ __forceinline__ int page_of(const Params& p, const Seg& g, int base, int lane) {
    const int j = base + (lane & 15);
    return j >= g.first && j < g.len ? __ldg(g.table + (j >> p.a.page_shift)) : 0;
  }
  // q's operand of k-steps 2 k2 and 2 k2 + 1 for rows 8 n .. 8 n + 7, part t
  static __device__ __forceinline__ void load_q4(uint32_t (&r)[4], uint32_t qaddr, int t, int n, int k2, int lane) {
    ldsm4(r, qaddr + (t * K::ROWS + 8 * n + (lane & 7)) * K::QB + (lane >> 3) * 16 + k2 * 64);
  }

  // Scores, weights and sums of one sub-tile in shared memory.  pos[n][e]: the position of the token of row 8 n +
  // 2 (lane & 3) + e; qs[n][e]: that row's factor from the raw product to log2 units (or to the cap's argument).
  template <bool CAREFUL>
  __device__ __forceinline__ void tile(const Params& p, const Seg& g, uint32_t stage, uint8_t* vrow, uint32_t qaddr,
                                       const uint32_t (&qreg)[K::QREG ? NT * K::NQ * (D / 32) : 1][4], int base,
                                       const int (&pos)[NT][2], const float (&qs)[NT][2], bool all, int lane) {
    const AttnArgs& a = p.a;
    float s[NT][4];  // positions base + lane / 4 (0, 1) and + 8 (2, 3)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
    // ---- scores
    const uint32_t kaddr = stage + (lane & 15) * K::RB + (lane >> 4) * 16;
#pragma unroll
    for (int k2 = 0; k2 < D / 32; ++k2) {
      uint32_t ka[2][4];
      if constexpr (K::F8) {
        uint32_t r[4];  // dims 0-15: positions 0-7, 8-15; dims 16-31 likewise
        ldsm4(r, kaddr + k2 * 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ka[h][0] = f8_pair(r[2 * h]);
          ka[h][1] = f8_pair(r[2 * h + 1]);
          ka[h][2] = f8_pair(r[2 * h] >> 16);
          ka[h][3] = f8_pair(r[2 * h + 1] >> 16);
        }
      } else {
        ldsm4(ka[0], kaddr + k2 * 64);
        ldsm4(ka[1], kaddr + k2 * 64 + 32);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        float(&acc)[4] = K::QF32 ? part : s[n];
#pragma unroll
        for (int t = 0; t < K::NQ; ++t) {
          if constexpr (K::QREG) {
            const uint32_t(&b)[4] = qreg[(n * K::NQ + t) * (D / 32) + k2];
            mma<K::F8>(acc, ka[0], b[0], b[1]);
            mma<K::F8>(acc, ka[1], b[2], b[3]);
          } else {
            uint32_t b[4];
            load_q4(b, qaddr, t, n, k2, lane);
            mma<K::F8>(acc, ka[0], b[0], b[1]);
            mma<K::F8>(acc, ka[1], b[2], b[3]);
          }
        }
        if constexpr (K::QF32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] += part[e];
        }
      }
    }
    // ---- weights
    const int j0 = base + (lane >> 2);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] *= qs[n][e & 1];
      if (a.softcap > 0.0f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = a.softcap * 1.4426950408889634f * tanhf(s[n][e]);
      }
      if (!all) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!sees<TREE>(j0 + 8 * (e >> 1), pos[n][e & 1], bits_of(n, e & 1, lane), g.len - a.T, a.window)) s[n][e] = -INFINITY;
        }
      }
      float mx[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(s[n][e], s[n][2 + e]);
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 4));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 8));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 16));
        mx[e] = fmaxf(mx[e], m[n][e]);
      }
      if (__any_sync(0xFFFFFFFFu, mx[0] != m[n][0] || mx[1] != m[n][1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float c = mx[e] == m[n][e] ? 1.0f : ex2(m[n][e] - mx[e]);
          l[n][e] *= c;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            o[n][d][e] *= c;
            o[n][d][2 + e] *= c;
          }
          m[n][e] = mx[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mm = m[n][e] == -INFINITY ? 0.0f : m[n][e];  // nothing seen yet: the weights are 0
        s[n][e] = ex2(s[n][e] - mm);
        s[n][2 + e] = ex2(s[n][2 + e] - mm);
        if constexpr (K::F8) {
          s[n][e] *= K::LIFT;
          s[n][2 + e] *= K::LIFT;
        }
        l[n][e] += s[n][e] + s[n][2 + e];
      }
    }
    if constexpr (CAREFUL) take_out(p, vrow, base, s, pos, lane);
    // ---- sums
    uint32_t w[NT][K::NP][2];  // positions 0-7 and 8-15, as the second operand
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = s[n][2 * h], y = s[n][2 * h + 1];
#pragma unroll
        for (int t = 0; t < K::NP; ++t) {
          const uint32_t v = pack2<K::F8>(x, y);
          const float2 b = unpack2<K::F8>(v);
          x -= b.x;
          y -= b.y;
          w[n][t][h] = transpose8(v);
        }
      }
    if constexpr (K::F8) {
      const uint32_t vaddr = stage + K::SUB + (lane & 15) * K::RB + (lane >> 4) * 16;
#pragma unroll
      for (int d2 = 0; d2 < D / 32; ++d2) {
        uint32_t r[4];  // dims 0-15: positions 0-7, 8-15; dims 16-31 likewise
        ldsm4t(r, vaddr + d2 * 32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t b0 = __byte_perm(r[2 * h], 0, 0x3120), b1 = __byte_perm(r[2 * h + 1], 0, 0x3120);
          const uint32_t va[4] = {f8_pair(b0), f8_pair(b0 >> 16), f8_pair(b1), f8_pair(b1 >> 16)};  // even dims, odd dims
#pragma unroll
          for (int n = 0; n < NT; ++n) add_product(o[n][2 * d2 + h], va, w[n]);
        }
      }
    } else {
      const uint32_t vaddr = stage + K::SUB + ((lane & 7) + (lane >> 4) * 8) * K::RB + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t va[4];
        ldsm4t(va, vaddr + d * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n) add_product(o[n][d], va, w[n]);
      }
    }
  }

  static __device__ __forceinline__ void add_product(float (&o)[4], const uint32_t (&va)[4], const uint32_t (&w)[K::NP][2]) {
    if constexpr (K::QF32) {
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < K::NP; ++t) mma<K::F8>(part, va, w[t][0], w[t][1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += part[e];
    } else {
#pragma unroll
      for (int t = 0; t < K::NP; ++t) mma<K::F8>(o, va, w[t][0], w[t][1]);
    }
  }

  // The dim of accumulator o[.][d][2 h + e].
  static __device__ __forceinline__ int dim_of(int d, int h, int lane) {
    return 16 * d + (K::F8 ? 2 * (lane >> 2) + h : (lane >> 2) + 8 * h);
  }
  static __device__ __forceinline__ float value_at(const uint8_t* row, int d) {
    if constexpr (K::F8) return static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(row)[d]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
  }
  __device__ __forceinline__ uint64_t bits_of(int n, int e, int lane) const {
    if constexpr (TREE) return this->tree[8 * n + 2 * (lane & 3) + e];
    else return 0;
  }
  __device__ __forceinline__ int new_from() const {
    if constexpr (TREE) return this->first_new;
    else return 0;
  }
  // Adds the values that are not finite to the rows that see them, and puts zeros in their place.
  __device__ __noinline__ void take_out(const Params& p, uint8_t* vrow, int base, const float (&s)[NT][4],
                                        const int (&pos)[NT][2], int lane) {
    for (int jj = 0; jj < WT; ++jj) {
      const int j = base + jj, from = (jj & 7) * 4 + (lane & 3);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float w = __shfl_sync(0xFFFFFFFFu, jj & 8 ? s[n][2 + e] : s[n][e], from);
          const bool seen = sees<TREE>(j, pos[n][e], bits_of(n, e, lane), new_from(), p.a.window);
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float v = value_at(vrow + jj * K::RB, dim_of(d, h, lane));
              if (seen && !finite(v)) o[n][d][2 * h + e] += w * v;
            }
        }
    }
    __syncwarp();
    for (int x = lane; x < WT * D; x += 32) {
      uint8_t* row = vrow + (x / D) * K::RB;
      if (!finite(value_at(row, x % D))) {
        if constexpr (K::F8) row[x % D] = 0;
        else reinterpret_cast<uint16_t*>(row)[x % D] = 0;
      }
    }
    __syncwarp();
  }

  // A warp's share of a segment: sub-tile `warp` of each tile.
  template <bool CAREFUL>
  __device__ __forceinline__ void run(const Params& p, const Seg& g, uint8_t* ring, uint32_t qaddr, const int (&pos)[NT][2],
                                      const float (&qs)[NT][2], int warp, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // a tree's padding rows: weights of 0 wherever masks are not looked at
        m[n][e] = TREE && pos[n][e] < 0 ? INFINITY : -INFINITY;
        l[n][e] = 0.0f;
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][d][e] = 0.0f;
    }
    const uint32_t rs = smem_u32(ring);
    const int n = g.t1 - g.t0, b0 = g.t0 * TK + warp * WT;
    int page = page_of(p, g, b0, lane);
#pragma unroll
    for (int i = 0; i < K::S; ++i) {
      const int next = i + 1 < n ? page_of(p, g, b0 + (i + 1) * TK, lane) : 0;
      if (i < n) issue(p, g, rs + i * K::STAGE, b0 + i * TK, page, lane);
      copy_commit();
      page = next;
    }
    uint32_t qreg[K::QREG ? NT * K::NQ * (D / 32) : 1][4];
    if constexpr (K::QREG) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < K::NQ; ++t)
#pragma unroll
          for (int k2 = 0; k2 < D / 32; ++k2) load_q4(qreg[(i * K::NQ + t) * (D / 32) + k2], qaddr, t, i, k2, lane);
    }
    // a sub-tile in [all_lo, all_hi] is seen by every row in full
    const int all_lo = p.a.window > 0 ? g.len - p.a.window : 0, all_hi = g.len - p.a.T - (TREE ? 1 : 0);
    int slot = 0;
    for (int i = 0; i < n; ++i) {
      const int base = b0 + i * TK;
      copy_wait<K::S - 1>();
      __syncwarp();
      const int next = i + K::S + 1 < n ? page_of(p, g, base + (K::S + 1) * TK, lane) : 0;
      if (base < g.len && base + WT > g.first)
        tile<CAREFUL>(p, g, rs + slot * K::STAGE, ring + slot * K::STAGE + K::SUB, qaddr, qreg, base, pos, qs,
                      base >= all_lo && base + WT - 1 <= all_hi, lane);
      __syncwarp();
      if (i + K::S < n) issue(p, g, rs + slot * K::STAGE, base + K::S * TK, page, lane);
      copy_commit();
      page = next;
      slot = slot + 1 == K::S ? 0 : slot + 1;
    }
    copy_wait<0>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[i][e] += __shfl_xor_sync(0xFFFFFFFFu, l[i][e], 4);
        l[i][e] += __shfl_xor_sync(0xFFFFFFFFu, l[i][e], 8);
        l[i][e] += __shfl_xor_sync(0xFFFFFFFFu, l[i][e], 16);
        if (TREE && pos[i][e] < 0) {  // whatever the keys were
          m[i][e] = -INFINITY;
          l[i][e] = 0.0f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[i][d][e] = o[i][d][2 + e] = 0.0f;
        }
      }
  }
  __device__ __forceinline__ bool all_finite() const {
    float x = 0.0f;  // a product with 0 keeps NaN and makes it of an infinity
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) x = fmaf(o[n][d][e], 0.0f, x);
    return __all_sync(0xFFFFFFFFu, x == 0.0f);
  }
};

__device__ __forceinline__ float4 load_q(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load_q(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  const float2 a = unpack2<false>(u.x), b = unpack2<false>(u.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

// q rows of an item as 16-bit parts in shared memory; rscale: each row's power of two (e4m3 cache).  A row is D / 4 lanes'
// work (D = 256: two rounds of a warp); a warp's rows are all loaded before the first is used.
template <class Q, class C, int D, int NT>
__device__ __forceinline__ void stage_q(const Params& p, uint8_t* qsm, float* rscale, int b, int hk, int r0, int warp, int lane) {
  using K = Cfg<Q, C, D, NT>;
  constexpr int LR = D < 128 ? D / 4 : 32, PR = D / 4 / LR;  // lanes per row, vectors per lane
  constexpr int RW = 32 / LR, N = (K::ROWS + NW * RW - 1) / (NW * RW);  // rows at a time per warp, times
  const AttnArgs& a = p.a;
  const int R = a.T * a.G;
  float4 x[N][PR];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int row = r0 + (n * NW + warp) * RW + lane / LR;
    if (row < R) {
      const int t = row / a.G, h = hk * a.G + row - t * a.G;
      const Q* src = static_cast<const Q*>(a.q) + (static_cast<int64_t>(b) * a.T + t) * a.q_stride + static_cast<int64_t>(h) * D;
#pragma unroll
      for (int i = 0; i < PR; ++i) x[n][i] = load_q(src + 4 * (lane % LR + i * LR));
    } else {
#pragma unroll
      for (int i = 0; i < PR; ++i) x[n][i] = make_float4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int r = (n * NW + warp) * RW + lane / LR;
    float back = 1.0f;
    if constexpr (K::F8) {
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < PR; ++i)
        mx = fmaxf(fmaxf(fmaxf(mx, fabsf(x[n][i].x)), fabsf(x[n][i].y)), fmaxf(fabsf(x[n][i].z), fabsf(x[n][i].w)));
#pragma unroll
      for (int d = LR / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
      // largest value into [2^13, 2^14); the factor and its inverse stay normal numbers
      const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 100);
      const float f = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
      back = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
#pragma unroll
      for (int i = 0; i < PR; ++i) x[n][i] = make_float4(x[n][i].x * f, x[n][i].y * f, x[n][i].z * f, x[n][i].w * f);
    }
    if (lane % LR == 0) rscale[r] = back;
#pragma unroll
    for (int i = 0; i < PR; ++i) {
      const int d = 4 * (lane % LR + i * LR);
      // e4m3: four neighbouring dims come in one register, so a k-step's slots hold them in this order
      const int s0 = K::F8 ? (d & ~15) + (d & 15) / 2 : d, s1 = K::F8 ? s0 + 8 : d + 2;
      float4 v = x[n][i];
#pragma unroll
      for (int t = 0; t < K::NQ; ++t) {
        uint8_t* row = qsm + (t * K::ROWS + r) * K::QB;
        const uint32_t w0 = pack2<K::F8>(v.x, v.y), w1 = pack2<K::F8>(v.z, v.w);
        *reinterpret_cast<uint32_t*>(row + 2 * s0) = w0;
        *reinterpret_cast<uint32_t*>(row + 2 * s1) = w1;
        const float2 b0 = unpack2<K::F8>(w0), b1 = unpack2<K::F8>(w1);
        v = make_float4(v.x - b0.x, v.y - b0.y, v.z - b1.x, v.w - b1.y);
      }
    }
  }
}

// ---- the line of tiles

// A sequence's length as its table allows, and the first position that some of its tokens sees.
__device__ __forceinline__ int length_of(const AttnArgs& a, int b, bool tell) {
  const int n = __ldg(a.seq_lens + b);
  if (n > a.room) {
    if (tell) record_error(a.err, DEV_ERR_PAGE);
    return a.room;
  }
  return max(n, 0);
}
__device__ __forceinline__ int first_of(const AttnArgs& a, int len) {
  return a.window > 0 ? max(0, len - a.T + 1 - a.window) : 0;
}
// Units of the line that one item of the sequence takes (an empty sequence has one, so that its rows are written).
template <int TILE = TK>
__device__ __forceinline__ int units_of(const AttnArgs& a, int len, int start) {
  return len > 0 ? start + (len + TILE - 1) / TILE - first_of(a, len) / TILE : 1;
}

// prefix [B + 1]: units (per head and row tile) before each sequence.  Threads 0 .. NTH - 1 work, every thread of the
// block calls.
template <int TILE = TK>
__device__ __forceinline__ void build_prefix(const AttnArgs& a, int start, int* prefix, int* s_scan) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.B + NTH - 1) / NTH;
  const int b0 = tid < NTH ? min(a.B, tid * per) : a.B, b1 = tid < NTH ? min(a.B, b0 + per) : a.B;
  int n = 0;
  for (int b = b0; b < b1; ++b) n += units_of<TILE>(a, length_of(a, b, blockIdx.x == 0), start);
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31 && tid < NTH) s_scan[warp] = incl;
  __syncthreads();
  int before = incl - n;
  for (int w = 0; w < warp && w < NW; ++w) before += s_scan[w];
  for (int b = b0; b < b1; ++b) {
    prefix[b] = before;
    before += units_of<TILE>(a, length_of(a, b, false), start);
    if (b == a.B - 1) prefix[a.B] = before;
  }
  __syncthreads();
}

// The line and its cut: ranges 0 .. nc - 1, `more` of share + 1 units, then of share.
struct Line {
  const int* prefix;
  int HR, nc, share, more;  // heads x row tiles of a sequence; ranges
  __device__ __forceinline__ Line(const AttnArgs& a, int RT, const int* pre) : Line(a, RT, pre, gridDim.x) {}
  __device__ __forceinline__ Line(const AttnArgs& a, int RT, const int* pre, int most) : prefix(pre) {
    HR = a.c.n_kv_heads * RT;  // the host has seen to it that the line's units fit 31 bits
    const int total = prefix[a.B] * HR;
    nc = min(total, most);
    share = total / nc;
    more = total - share * nc;
  }
  __device__ __forceinline__ int bound(int k) const { return k * share + min(k, more); }
  __device__ __forceinline__ int range_of(int u) const {
    return u < more * (share + 1) ? u / (share + 1) : more + (u - more * (share + 1)) / share;
  }
};
// The item that unit u is of: its tiles are units [i0, i1).
struct Item {
  int b, hr, hk, rt, len, i0, i1;
  __device__ __forceinline__ Item(const AttnArgs& a, const Line& line, int RT, int start, int u) {
    b = 0;  // the last sequence that starts at or before u
    for (int w = 1 << (31 - __clz(a.B)); w > 0; w >>= 1)
      if (b + w < a.B && line.prefix[b + w] * line.HR <= u) b += w;
    const int nt = line.prefix[b + 1] - line.prefix[b];
    hr = (u - line.prefix[b] * line.HR) / nt;
    hk = hr / RT;
    rt = hr - hk * RT;
    len = length_of(a, b, false);
    i1 = line.prefix[b] * line.HR + (hr + 1) * nt;
    i0 = len > 0 ? i1 - nt + start : i1 - 1;
  }
};

// By one thread of the range that has the item's first tile.
__device__ __forceinline__ void note_split(Split* split, int by_item, const Line& line, const Item& it, int range, bool whole, int slot) {
  const int item = it.b * line.HR + it.hr;
  if (!whole) split[by_item ? item : range] = {item, range, line.range_of(it.i1 - 1) - range + 1, slot};
  else if (by_item) split[item].parts = 0;
}

// The last CTA to arrive with its part of an item joins the ranges' sums: NTH threads (tid) call with their part stored,
// sync being their barrier.  scratch: `room` bytes of shared memory; s_sum, s_i, s_last: shared.  write(r, d, sum, factor).
template <int D, int ROWS, class Sync, class Write>
__device__ __forceinline__ void join_parts(const Params& p, const Line& line, const Item& it, int R, int tid, float* factor, int room,
                                           float* s_sum, float* s_i, int* s_last, Sync sync, Write write) {
  const int warp = tid >> 5, lane = tid & 31;
  const int ca = line.range_of(it.i0), cb = line.range_of(it.i1 - 1);
  const int parts = cb - ca + 1;  // the item's tiles lie in ranges ca .. cb
  sync();
  if (tid == 0) {
    __threadfence();  // after the barrier: orders the whole block's stores before the arrival
    int* cnt = p.count + ca;  // no two split items begin in one range: the first one goes on past its end
    *s_last = atomicAdd(cnt, 1) == parts - 1;
    if (*s_last) *cnt = 0;
  }
  sync();
  if (!*s_last) return;
  __threadfence();
  // every range but the first starts in the item's tiles
  const int slot0 = 2 * ca + (line.bound(ca) >= it.i0 ? 1 : 0);
  auto slot_of = [&](int k) { return k == 0 ? slot0 : 2 * (ca + k) + 1; };
  const int fit = min(R, room / 4 / parts);  // factor: [parts][rows], as many rows at a time as fit
  for (int rb = 0; rb < R; rb += fit) {
    const int rows = min(fit, R - rb);
    // a row's parts are spread over as many lanes as they need, so that a warp takes several rows at a time
    const int span = parts >= 32 ? 32 : 1 << (32 - __clz(parts - 1)), k0 = lane & (span - 1);
    for (int r1 = warp * (32 / span); r1 < rows; r1 += NW * (32 / span)) {
      const int r = r1 + lane / span;
      float mm = -INFINITY, ll = 0.0f;
      if (r < rows)
        for (int k = k0; k < parts; k += span) {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (static_cast<int64_t>(slot_of(k)) * ROWS + rb + r) * 2));
          factor[k * rows + r] = x.x;
          mm = fmaxf(mm, x.x);
          if (parts <= 32) ll = x.y;
        }
      for (int o = span / 2; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
      const float ms = mm == -INFINITY ? 0.0f : mm;
      if (r < rows) {
        const float first = ll;
        ll = 0.0f;
        for (int k = k0; k < parts; k += span) {
          const float e = ex2(factor[k * rows + r] - ms);
          factor[k * rows + r] = e;
          ll += e * (parts <= 32 ? first : __ldcg(p.part_ml + (static_cast<int64_t>(slot_of(k)) * ROWS + rb + r) * 2 + 1));
        }
      }
      for (int o = span / 2; o > 0; o >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, o);
      if (r < rows && k0 == 0) s_i[r] = ll == 0.0f ? 0.0f : p.a.c.v_scale / ll;
    }
    sync();
    // Vectors of the rows, four at a time per lane, over the parts, two in flight.  Few parts: every warp takes all of them
    // for its vectors; many: each warp a quarter of them for all vectors, joined in shared memory.
    constexpr int XU = 4;
    const int vecs = rows * (D / 4), groups = parts > 8 ? NW : 1, warps = NW / groups;
    float4* sum = reinterpret_cast<float4*>(s_sum);
    for (int x1 = 0; x1 < vecs; x1 += warps * 32 * XU) {
      const int x0 = x1 + (groups == 1 ? warp * 32 : 0) + lane;
      float4 acc[XU];
#pragma unroll
      for (int i = 0; i < XU; ++i) acc[i] = make_float4(0, 0, 0, 0);
#pragma unroll 2
      for (int k = groups == 1 ? 0 : warp; k < parts; k += groups) {
        const float4* part = reinterpret_cast<const float4*>(p.part + (static_cast<int64_t>(slot_of(k)) * ROWS + rb) * D);
#pragma unroll
        for (int i = 0; i < XU; ++i) {
          const int x = x0 + i * warps * 32;
          if (x < vecs) add4(acc[i], factor[k * rows + x / (D / 4)], __ldcg(part + x));
        }
      }
      if (groups > 1) {
#pragma unroll
        for (int i = 0; i < XU; ++i) sum[(warp * XU + i) * 32 + lane] = acc[i];
        sync();
        if (warp < XU) {
          acc[0] = sum[warp * 32 + lane];
#pragma unroll
          for (int w = 1; w < NW; ++w) add4(acc[0], 1.0f, sum[(w * XU + warp) * 32 + lane]);
          const int x = x0 + warp * 32;
          if (x < vecs) write(rb + x / (D / 4), 4 * (x % (D / 4)), acc[0], s_i[x / (D / 4)]);
        }
        sync();
      } else {
#pragma unroll
        for (int i = 0; i < XU; ++i) {
          const int x = x0 + i * warps * 32;
          if (x < vecs) write(rb + x / (D / 4), 4 * (x % (D / 4)), acc[i], s_i[x / (D / 4)]);
        }
      }
    }
    sync();
  }
}
constexpr int JOIN_SUMS = NW * 4 * 32 * 4;  // floats of s_sum

template <class Q, class C, int D, int NT, bool TREE>
__global__ void __launch_bounds__(NTH, (Cfg<Q, C, D, NT>::CPS)) attn_kernel(const __grid_constant__ Params p) {
  using K = Cfg<Q, C, D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Scratch scratch;
  float* rscale = reinterpret_cast<float*>(smem);  // [ROWS]
  float* s_i = rscale + K::ROWS;                   // [ROWS] the join's 1 / weight sum
  float* w_ml = s_i + K::ROWS;                     // [NW][ROWS][2] each warp's maximum and weight sum
  uint8_t* qsm = smem + K::HDR;
  uint8_t* ring = smem + K::FIXED;
  const AttnArgs& a = p.a;
  int* prefix = reinterpret_cast<int*>(ring + K::RING);  // [B + 1] tiles before each sequence
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();

  build_prefix(a, START, prefix, scratch.scan);
  const Line line(a, p.RT, prefix);
  const int range = blockIdx.x;
  if (range >= line.nc) {
    if (TREE && threadIdx.x == 0 && !p.by_item) p.split[range].parts = 0;
    return;
  }
  const int lo = line.bound(range), hi = line.bound(range + 1);
  if (TREE && threadIdx.x == 0 && !p.by_item) p.split[range].parts = 0;
  for (int u = lo; u < hi;) {
    const Item it(a, line, p.RT, START, u);
    const int end = min(it.i1, hi);
    if (u < it.i0) u = it.i0;
    if (u >= end) {  // none of its tiles is in this range
      u = end;
      continue;
    }
    const int r0 = it.rt * K::ROWS, R = min(K::ROWS, a.T * a.G - r0);
    auto write = [&](int r, int d, float4 v, float inv) {
      const int row = r0 + r, t = row / a.G, h = it.hk * a.G + row - t * a.G;
      put4(static_cast<Q*>(a.out) + ((static_cast<int64_t>(it.b) * a.T + t) * a.Hq + h) * D + d, v, inv);
    };
    if (it.len == 0) {
      if (TREE && threadIdx.x == 0) note_split(p.split, p.by_item, line, it, range, true, 0);
      for (int x = threadIdx.x; x < R * (D / 4); x += NTH) write(x / (D / 4), 4 * (x % (D / 4)), make_float4(0, 0, 0, 0), 0.0f);
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

    stage_q<Q, C, D, NT>(p, qsm, rscale, it.b, it.hk, r0, warp, lane);
    __shared__ TreeRows<TREE ? K::ROWS : 1> rows;  // (a chain's kernels have none)
    if (TREE && warp == 0) {
      const TreeToken x(a, it.b, min((r0 + lane) / a.G, a.T - 1), g.len);
      if (lane < K::ROWS) {
        rows.bits[lane] = x.bits;
        rows.pos[lane] = x.pos;
      }
    }
    __syncthreads();
    int pos[NT][2];
    float qs[NT][2];
    const float f = a.scale * a.c.k_scale * (a.softcap > 0.0f ? 1.0f / a.softcap : 1.4426950408889634f);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * (lane & 3) + e;
        if constexpr (TREE) pos[n][e] = rows.pos[r];
        else pos[n][e] = g.len - a.T + min((r0 + r) / a.G, a.T - 1);
        qs[n][e] = f * rscale[r];
      }
    Warp<Q, C, D, NT, TREE> w;
    if constexpr (TREE) w.tree = rows.bits, w.first_new = g.len - a.T;
    uint8_t* mine = ring + warp * (K::S * K::STAGE);
    w.template run<false>(p, g, mine, smem_u32(qsm), pos, qs, warp, lane);
    if (!w.all_finite()) {
      Warp<Q, C, D, NT, TREE> again;  // an object of its own: the call in it keeps this one out of registers
      if constexpr (TREE) again.tree = rows.bits, again.first_new = g.len - a.T;
      again.template run<true>(p, g, mine, smem_u32(qsm), pos, qs, warp, lane);
      w = again;
    }

    // ---- the warps' sums, side by side in the ring's place
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * (lane & 3) + e;
        if (lane < 4) {
          w_ml[(warp * K::ROWS + r) * 2] = w.m[n][e];
          w_ml[(warp * K::ROWS + r) * 2 + 1] = w.l[n][e];
        }
        float* so = reinterpret_cast<float*>(mine + r * K::OB);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          if constexpr (K::F8) {
            *reinterpret_cast<float2*>(so + w.dim_of(d, 0, lane)) = make_float2(w.o[n][d][e], w.o[n][d][2 + e]);
          } else {
            so[w.dim_of(d, 0, lane)] = w.o[n][d][e];
            so[w.dim_of(d, 1, lane)] = w.o[n][d][2 + e];
          }
        }
      }
    __syncthreads();
    const bool whole = u == it.i0 && end == it.i1;
    const int slot = 2 * range + (lo >= it.i0 ? 1 : 0);  // the range starts in these tiles (1), or before them
    for (int x = threadIdx.x; x < R * (D / 4); x += NTH) {
      const int r = x / (D / 4), d = 4 * (x % (D / 4));
      float mm = -INFINITY, ll = 0.0f;
      float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < NW; ++k) mm = fmaxf(mm, w_ml[(k * K::ROWS + r) * 2]);
      const float ms = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float e = ex2(w_ml[(k * K::ROWS + r) * 2] - ms);
        ll += w_ml[(k * K::ROWS + r) * 2 + 1] * e;
        add4(acc, e, *reinterpret_cast<const float4*>(ring + k * (K::S * K::STAGE) + r * K::OB + d * 4));
      }
      if (whole) {
        write(r, d, acc, ll == 0.0f ? 0.0f : a.c.v_scale / ll);
      } else {
        *reinterpret_cast<float4*>(p.part + (static_cast<int64_t>(slot) * K::ROWS + r) * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(slot) * K::ROWS + r) * 2) = make_float2(mm, ll);
      }
    }
    if constexpr (TREE) {
      if (u == it.i0 && threadIdx.x == 0) note_split(p.split, p.by_item, line, it, range, whole, slot);
    } else if (!whole) {  // in the ring's place, too
      constexpr int ROOM = K::RING - JOIN_SUMS * 4;
      join_parts<D, K::ROWS>(p, line, it, R, threadIdx.x, reinterpret_cast<float*>(ring), ROOM, reinterpret_cast<float*>(ring + ROOM),
                             s_i, &scratch.last, [] { __syncthreads(); }, write);
    }
    __syncthreads();
    u = end;
  }
}

template <class Q, class C, int D, int NT, bool TREE>
cudaError_t launch_one(const Params& p, cudaStream_t st, AttnShape* ask) {
  using K = Cfg<Q, C, D, NT>;
  const size_t smem = K::SMEM + 4 * (static_cast<size_t>(p.a.B) + 1);
  static size_t fits[64] = {0};  // shared memory with which CPS CTAs are known to be resident, per device
  static bool set[64] = {false};
  const int dev = current_device_id();
  if (!set[dev]) {  // for all calls: one at the same time may want less
    constexpr int most = K::SMEM + 4 * (kMaxSeqs + 1);
    static_assert(most + 2048 <= kMaxSmemPerBlock, "beside the static memory");
    const cudaError_t e = cudaFuncSetAttribute(attn_kernel<Q, C, D, NT, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  // one range per CTA, all of them resident: one that waits for another's place would start when that one has ended
  int ctas = K::CPS;
  if (K::CPS > 1 && smem > fits[dev]) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, attn_kernel<Q, C, D, NT, TREE>, NTH, smem);
    if (e != cudaSuccess) return e;
    if (ctas >= K::CPS) fits[dev] = smem;
    ctas = ctas < 1 ? 1 : ctas < K::CPS ? ctas : K::CPS;
  }
  if (ask) {
    ask->planned = K::CPS;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ask->resident, attn_kernel<Q, C, D, NT, TREE>, NTH, smem);
  }
  // no more ranges than units that sequences as long as the table can have: CTAs without one only take their places (one of
  // 1000 positions: 9.4 us in place of 9.6)
  const int64_t units = (START + (static_cast<int64_t>(p.a.room) + TK - 1) / TK) * p.a.B * p.a.c.n_kv_heads * p.RT;
  const int grid = static_cast<int>(min_i64(num_sms() * ctas, units));
  if constexpr (TREE) {
    const cudaError_t e = launch_pdl(attn_kernel<Q, C, D, NT, TREE>, dim3(grid), dim3(NTH), smem, st, p);
    return e != cudaSuccess ? e : launch_tree_join(p, K::ROWS, D, sizeof(Q) == 4, grid, st);
  }
  return launch_pdl(attn_kernel<Q, C, D, NT, TREE>, dim3(grid), dim3(NTH), smem, st, p);
}

template <class Q, class C, bool TREE = false>
cudaError_t launch_kind(const Params& p, int rows, cudaStream_t st, AttnShape* ask) {
  switch (p.a.c.head_dim * 100 + rows) {
    case 6408: return launch_one<Q, C, 64, 1, TREE>(p, st, ask);
    case 6416: return launch_one<Q, C, 64, 2, TREE>(p, st, ask);
    case 6432: return launch_one<Q, C, 64, 4, TREE>(p, st, ask);
    case 12808: return launch_one<Q, C, 128, 1, TREE>(p, st, ask);
    case 12816: return launch_one<Q, C, 128, 2, TREE>(p, st, ask);
    case 12832: return launch_one<Q, C, 128, 4, TREE>(p, st, ask);
    case 25608: return launch_one<Q, C, 256, 1, TREE>(p, st, ask);
    default: return launch_one<Q, C, 256, 2, TREE>(p, st, ask);
  }
}

}  // namespace attn

// More than 16 rows, bf16 q and cache, heads of 64 or 128 values (kq_attn_wide.cu).
constexpr int kWideRows = 128;
cudaError_t launch_attn_wide(const attn::Params& p, cudaStream_t st, AttnShape* ask);

// One translation unit per cache and query type (rows: query rows per pass, 8, 16 or 32).
cudaError_t launch_attn_bf16_bf16(const attn::Params& p, int rows, cudaStream_t st, AttnShape* ask);
cudaError_t launch_attn_bf16_f32(const attn::Params& p, int rows, cudaStream_t st, AttnShape* ask);
cudaError_t launch_attn_f8_bf16(const attn::Params& p, int rows, cudaStream_t st, AttnShape* ask);
cudaError_t launch_attn_f8_f32(const attn::Params& p, int rows, cudaStream_t st, AttnShape* ask);
// Trees of drafted tokens (kq_attn_tree_<cache>_<query>.cu).
cudaError_t launch_attn_tree_bf16_bf16(const attn::Params& p, int rows, cudaStream_t st);
cudaError_t launch_attn_tree_bf16_f32(const attn::Params& p, int rows, cudaStream_t st);
cudaError_t launch_attn_tree_f8_bf16(const attn::Params& p, int rows, cudaStream_t st);
cudaError_t launch_attn_tree_f8_f32(const attn::Params& p, int rows, cudaStream_t st);

}  // namespace kq
