// kq_sample.cu -- the next token of each row of logits, from a given uniform
// number u:  w_i = exp((l_i - l_max) / temperature); the words in descending
// order of their logits (equal ones by index), cut to top_k, then to the
// shortest prefix that holds top_p of the remaining weight, then to the words
// with w_i >= min_p; the token is the first word whose running sum of the kept
// weights exceeds u times their total.
//
// Weights are summed as integers, w_i in units of 2^-40 of the largest: the
// sums are exact, so no order of summation changes a cut or the token (what a
// word below 2^-41 of the likeliest loses is far below the fp32 rounding of
// the likeliest itself), and 2^20 words stay below 2^60.
//
// Bound: each logit is read once from memory (bytes), and behind that a chain
// of dependent steps per row (latency).  A row is a cluster of up to 8 CTAs.
//  * One pass finds each thread's largest logit, and from the threads' largest
//    ones a threshold with at least as many words above it as the row needs
//    (top_k of them, else 64); the few words above it are listed.  No CTA
//    waits for another up to here.  Only a row without top_k takes a second
//    pass (from L2): its total weight.
//  * The first CTA sorts the lists and makes the cuts and the choice on the
//    sorted prefix.  Words it lists are complete above the highest threshold,
//    so whatever falls inside is final.
//  * A row whose cut or token falls outside (flat distributions, large top_k)
//    goes on with histograms of counts and weights over the whole row, 1024
//    bins at a time, until the words of the bin that holds the answer fit the
//    list; equal logits are told apart by index as further digits of the
//    sorting key.
#include "kq_cache.h"

namespace kq {
namespace {

constexpr int STH = 512;      // threads per CTA
constexpr int SW = STH / 32;
constexpr int CAND = 1024;    // words a CTA lists
constexpr int LIST = 2048;    // words the first CTA sorts
constexpr int BINS = 1024;
constexpr int TOPK_FAST = 256;  // top_k up to here by thresholds (of 512 threads' largest logits)
constexpr float kSpan = 29.0f;  // exp(-29) < 2^-41: words this far below the largest weigh nothing
constexpr int kIdxBits = 20;

struct Cmd {  // from the first CTA to the others
  int done;
  int bin0, shift;  // the words looked at: of level-0 bin `bin0` (-1: all), with the key digits above shift + 10 of `pre`
  unsigned long long pre;
  int gather;       // list the words of digit `pre >> shift` (level 0: of bin0)
};

struct Smem {
  uint32_t count[BINS], limb[3][BINS];
  unsigned long long list[LIST];
  unsigned long long cand[CAND];
  unsigned long long scan_m[SW], red_m[SW];
  int scan_c[SW];
  float red_f[SW];
  unsigned long long mass;      // this CTA's sum
  unsigned long long tau;       // its threshold, as the largest sorting key that is listed for sure
  int ncand, nlist, overflow;
  float bmax;
  Cmd cmd;
  unsigned long long found_cv, found_before;  // locate()'s answer
  int pick, pick_c;
  unsigned long long pick_m;
};

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ float one(const float* p) { return __ldg(p); }
__device__ __forceinline__ float one(const __nv_bfloat16* p) {
  return bf16_lo(__ldg(reinterpret_cast<const unsigned short*>(p)));
}
template <class F>
__device__ __forceinline__ void each4(const float*, uint4 v, int i, F f) {
  f(i, __uint_as_float(v.x)), f(i + 1, __uint_as_float(v.y)), f(i + 2, __uint_as_float(v.z)), f(i + 3, __uint_as_float(v.w));
}
template <class F>
__device__ __forceinline__ void each4(const __nv_bfloat16*, uint4 v, int i, F f) {
  f(i, bf16_lo(v.x)), f(i + 1, bf16_hi(v.x)), f(i + 2, bf16_lo(v.y)), f(i + 3, bf16_hi(v.y));
  f(i + 4, bf16_lo(v.z)), f(i + 5, bf16_hi(v.z)), f(i + 6, bf16_lo(v.w)), f(i + 7, bf16_hi(v.w));
}

// f(index, logit) for every word of this CTA's share of the row: 16-byte chunks by address, single loads where a chunk
// reaches past the row.
template <class X, class F>
__device__ __forceinline__ void each_word(const X* row, int V, int rank, int CS, F f) {
  constexpr int E = 16 / static_cast<int>(sizeof(X)), U = 4;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(X)) % E);
  const int n = (V + off + E - 1) / E, step = CS * STH;
  for (int c0 = rank * STH + static_cast<int>(threadIdx.x); c0 < n; c0 += U * step) {
    uint4 v[U];
    bool full[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = (c0 + k * step) * E - off;
      full[k] = i >= 0 && i + E <= V;
      if (full[k]) v[k] = __ldg(reinterpret_cast<const uint4*>(row + i));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = (c0 + k * step) * E - off;
      if (full[k]) {
        each4(row, v[k], i, f);
      } else if (c0 + k * step < n) {
        for (int j = max(i, 0); j < min(i + E, V); ++j) f(j, one(row + j));
      }
    }
  }
}

// Words compare by their sorting key, ascending: the logit's bits in an order that compares as integers, inverted, then
// the index.  -0 counts as 0.
__device__ __forceinline__ unsigned long long sort_key(float x, int i) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t up = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(~up) << kIdxBits) | static_cast<uint32_t>(i);
}
__device__ __forceinline__ float logit_of(unsigned long long cv) {
  const uint32_t up = ~static_cast<uint32_t>(cv >> kIdxBits);
  return __uint_as_float(up & 0x80000000u ? up & 0x7FFFFFFFu : ~up);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct Row {
  float lmax, c;  // c = log2(e) / temperature
  float zs;       // level-0 bins per unit of logit
  __device__ __forceinline__ float weight(float l) const { return l == lmax ? 1.0f : ex2((l - lmax) * c); }
  // the weight in units of 2^-40 as 2^20 hi + lo, |lo| <= 2^19 (adding 1.5 * 2^23 rounds to an integer)
  __device__ __forceinline__ void parts(float l, int& hi, int& lo) const {
    const float w = weight(l) * 1048576.0f;  // NaN (a NaN logit) is taken out by the caller
    const float h = w + 12582912.0f;
    hi = __float_as_int(h) - 0x4B400000;
    lo = __float_as_int(fmaf(w - (h - 12582912.0f), 1048576.0f, 12582912.0f)) - 0x4B400000;
  }
  __device__ __forceinline__ unsigned long long units(float l) const {
    int hi, lo;
    parts(l, hi, lo);
    return static_cast<unsigned long long>((static_cast<long long>(hi) << 20) + lo);
  }
  __device__ __forceinline__ int bin(float l) const {
    return l == lmax ? 0 : static_cast<int>(fminf((lmax - l) * zs, static_cast<float>(BINS - 1)));
  }
};

// ---- block-wide helpers (every thread calls them)
__device__ __forceinline__ unsigned long long block_sum(Smem& s, unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red_m[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < SW; ++i) v += s.red_m[i];
  return v;
}
// Exclusive prefix over the threads.
__device__ __forceinline__ void block_scan(Smem& s, unsigned long long& m, int& c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long im = m;
  int ic = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long tm = __shfl_up_sync(0xFFFFFFFFu, im, o);
    const int tc = __shfl_up_sync(0xFFFFFFFFu, ic, o);
    if (lane >= o) { im += tm; ic += tc; }
  }
  __syncthreads();
  if (lane == 31) { s.scan_m[warp] = im; s.scan_c[warp] = ic; }
  __syncthreads();
  im -= m;
  ic -= c;
  for (int w = 0; w < warp; ++w) { im += s.scan_m[w]; ic += s.scan_c[w]; }
  m = im;
  c = ic;
}
// Sorts s.list[0, n) ascending, n <= LIST.
__device__ void sort_list(Smem& s, int n) {
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += STH) s.list[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < size / 2; t += STH) {
        const int i = 2 * t - (t & (j - 1)), x = i + j;  // i has bit j clear
        const unsigned long long a = s.list[i], b = s.list[x];
        if ((a > b) == ((i & k) == 0)) { s.list[i] = b; s.list[x] = a; }
      }
      __syncthreads();
    }
}

// ---- another CTA's shared memory
template <class T>
__device__ __forceinline__ uint32_t at_rank(const T* p, int rank) {
  return cluster_map(smem_u32(p), static_cast<uint32_t>(rank));
}
__device__ __forceinline__ uint32_t peer32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ unsigned long long peer64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ int peer_add(uint32_t addr, int v) {
  int r;
  asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(r) : "r"(addr), "r"(v) : "memory");
  return r;
}

// The four words of the sorted list that thread t holds, and what lies before them.
struct Held {
  unsigned long long cv[LIST / STH], w[LIST / STH], before;
  int n;
};
__device__ __forceinline__ Held hold(Smem& s, const Row& r, int n) {
  Held h;
  unsigned long long m = 0;
  int c = 0;
  h.n = 0;
#pragma unroll
  for (int i = 0; i < LIST / STH; ++i) {
    const int j = static_cast<int>(threadIdx.x) * (LIST / STH) + i;
    h.cv[i] = j < n ? s.list[j] : 0;
    h.w[i] = j < n ? r.units(logit_of(h.cv[i])) : 0;
    m += h.w[i];
    h.n += j < n;
  }
  block_scan(s, m, c);
  h.before = m;
  return h;
}
// The held word at which the running sum passes x: s.found_cv, s.found_before and s.pick (its place, else -1).
__device__ __forceinline__ bool pass_at(Smem& s, const Held& h, unsigned long long base, unsigned long long x) {
  __syncthreads();
  if (threadIdx.x == 0) s.pick = -1;
  __syncthreads();
  unsigned long long c = base + h.before;
#pragma unroll
  for (int i = 0; i < LIST / STH; ++i) {
    if (c <= x && x < c + h.w[i]) {
      s.found_cv = h.cv[i];
      s.found_before = c;
      s.pick = static_cast<int>(threadIdx.x) * (LIST / STH) + i;
    }
    c += h.w[i];
  }
  __syncthreads();
  return s.pick >= 0;
}

// Over the whole row, every CTA of the cluster: the word at which the running sum of weights (by_count: of words)
// passes x; found_cv and found_before (the weight before it) in the first CTA, false there when there is none.
template <class X>
__device__ bool locate(Smem& s, const X* row, int V, int rank, int CS, const Row& r, unsigned long long x, bool by_count) {
  unsigned long long base_m = 0, base_c = 0;
  if (threadIdx.x == 0 && rank == 0) {
    s.cmd.bin0 = -1;
    s.cmd.shift = 0;
    s.cmd.pre = 0;
    s.cmd.gather = 0;
  }
  bool found = true;
  for (;;) {
    if (threadIdx.x == 0) s.nlist = 0;
    cluster_sync();  // the command is written, the first CTA's list is empty, and it is done with the histograms
    for (int i = threadIdx.x; i < BINS; i += STH) { s.count[i] = 0; s.limb[0][i] = 0; s.limb[1][i] = 0; s.limb[2][i] = 0; }
    __syncthreads();
    const int bin0 = static_cast<int>(peer32(at_rank(&s.cmd.bin0, 0)));
    const int shift = static_cast<int>(peer32(at_rank(&s.cmd.shift, 0)));
    const int gather = static_cast<int>(peer32(at_rank(&s.cmd.gather, 0)));
    const unsigned long long pre = peer64(at_rank(&s.cmd.pre, 0));
    if (gather == 2) {
      cluster_sync();  // every CTA has read the command
      break;
    }
    const uint32_t list0 = at_rank(s.list, 0), nlist0 = at_rank(&s.nlist, 0);
    each_word(row, V, rank, CS, [&](int i, float l) {
      if (!(l > -INFINITY)) return;
      const unsigned long long w = r.units(l);
      if (w == 0) return;
      const int b = r.bin(l);
      int d = b;
      if (bin0 >= 0) {
        if (b != bin0) return;
        const unsigned long long cv = sort_key(l, i);
        if (gather) {
          if (shift < 64 && (cv >> shift) != (pre >> shift)) return;
          const int at = peer_add(nlist0, 1);
          if (at < LIST) peer_store64(list0 + 8 * at, cv);
          return;
        }
        if (shift + 10 < 52 && (cv >> (shift + 10)) != (pre >> (shift + 10))) return;
        d = static_cast<int>(cv >> shift) & (BINS - 1);
      }
      atomicAdd(&s.count[d], 1u);
      atomicAdd(&s.limb[0][d], static_cast<uint32_t>(w) & 0x3FFFu);
      atomicAdd(&s.limb[1][d], static_cast<uint32_t>(w >> 14) & 0x3FFFu);
      atomicAdd(&s.limb[2][d], static_cast<uint32_t>(w >> 28));
    });
    cluster_sync();
    if (rank != 0) continue;
    if (gather) {
      const int n = min(s.nlist, LIST);
      sort_list(s, n);
      if (by_count) {  // the place in the list is known
        const int at = static_cast<int>(x - base_c);
        const Held h = hold(s, r, n);
        unsigned long long c = base_m + h.before;
#pragma unroll
        for (int i = 0; i < LIST / STH; ++i) {
          if (static_cast<int>(threadIdx.x) * (LIST / STH) + i == at) { s.found_cv = h.cv[i]; s.found_before = c; }
          c += h.w[i];
        }
        __syncthreads();
      } else {
        pass_at(s, hold(s, r, n), base_m, x);
      }
      if (threadIdx.x == 0) s.cmd.gather = 2;
      continue;
    }
    // the cluster's histogram: two neighbouring bins per thread
    unsigned long long m[2] = {0, 0};
    int c[2] = {0, 0};
    for (int k = 0; k < CS; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int b = 2 * threadIdx.x + e;
        c[e] += static_cast<int>(peer32(at_rank(&s.count[b], k)));
        m[e] += static_cast<unsigned long long>(peer32(at_rank(&s.limb[0][b], k))) +
                (static_cast<unsigned long long>(peer32(at_rank(&s.limb[1][b], k))) << 14) +
                (static_cast<unsigned long long>(peer32(at_rank(&s.limb[2][b], k))) << 28);
      }
    unsigned long long pm = m[0] + m[1];
    int pc = c[0] + c[1];
    block_scan(s, pm, pc);
    __syncthreads();
    if (threadIdx.x == 0) s.pick = -1;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const unsigned long long before = by_count ? base_c + pc : base_m + pm, in = by_count ? c[e] : m[e];
      if (before <= x && x < before + in) {
        s.pick = 2 * threadIdx.x + e;
        s.pick_m = base_m + pm;
        s.pick_c = static_cast<int>(base_c) + pc;
        s.nlist = c[e];
      }
      pm += m[e];
      pc += c[e];
    }
    __syncthreads();
    const int pick = s.pick, in_bin = s.nlist;
    if (pick >= 0) { base_m = s.pick_m; base_c = s.pick_c; }
    __syncthreads();
    if (threadIdx.x == 0) {
      if (pick < 0) {
        s.cmd.gather = 2;
      } else if (bin0 < 0) {
        s.cmd.bin0 = pick;
        s.cmd.shift = in_bin <= LIST ? 64 : 42;
        s.cmd.gather = in_bin <= LIST;
      } else {
        const unsigned long long p = (shift + 10 < 52 ? pre >> (shift + 10) << (shift + 10) : 0) |
                                     (static_cast<unsigned long long>(pick) << shift);
        s.cmd.pre = p;
        s.cmd.gather = in_bin <= LIST;
        if (in_bin > LIST) s.cmd.shift = shift - 10;
      }
    }
    found = pick >= 0;
    __syncthreads();
  }
  return found;
}

template <class X>
__global__ void __launch_bounds__(STH, 2) sample_kernel(const __grid_constant__ SampleArgs a, int CS) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = blockIdx.x / CS, rank = blockIdx.x - m * CS, V = a.V;
  const X* row = static_cast<const X*>(a.logits) + m * a.row_stride;
  float temp = a.temperature ? __ldg(a.temperature + m) : 1.0f;
  int k = a.top_k ? __ldg(a.top_k + m) : 0;
  if (!(temp > 0.0f)) {  // the largest logit
    temp = 1.0f;
    k = 1;
  }
  if (k < 0 || k >= V) k = 0;
  const float p = a.top_p ? __ldg(a.top_p + m) : 1.0f, mp = a.min_p ? __ldg(a.min_p + m) : 0.0f;
  const float u = __ldg(a.u + m);

  // ---- this CTA's words above its threshold
  if (tid == 0) { s.ncand = 0; s.overflow = 0; s.tau = 0; s.cmd.done = 0; }
  for (int i = tid; i < BINS; i += STH) s.count[i] = 0;
  float mine = -INFINITY;
  each_word(row, V, rank, CS, [&](int, float l) { mine = fmaxf(mine, l); });
  float mx = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) s.red_f[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SW; ++i) mx = fmaxf(mx, s.red_f[i]);
  Row r;
  r.lmax = mx;
  r.c = 1.4426950408889634f / temp;
  r.zs = static_cast<float>(BINS) / kSpan / temp;
  const int want = k > 0 && k <= TOPK_FAST ? max(k, 16) : 64;
  const bool some = mine > -INFINITY && (mine == mx || (mx - mine) * r.zs < static_cast<float>(BINS));
  const int bin = some ? r.bin(mine) : BINS;
  if (some) atomicAdd(&s.count[bin], 1u);
  __syncthreads();
  {
    unsigned long long none = 0;
    const int c0 = s.count[2 * tid], c1 = s.count[2 * tid + 1];
    int before = c0 + c1;
    block_scan(s, none, before);
    if (tid == 0) s.pick = BINS;  // all of them: the list is complete
    __syncthreads();
    if (before < want && before + c0 >= want) s.pick = 2 * tid;
    else if (before + c0 < want && before + c0 + c1 >= want) s.pick = 2 * tid + 1;
    __syncthreads();
  }
  const int last = s.pick;
  // the threshold: the smallest of the threads' largest logits in the bins up to `last`, or what weighs anything
  float cut = INFINITY;
  if (last < BINS) {
    if (some && bin <= last) cut = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cut = fminf(cut, __shfl_xor_sync(0xFFFFFFFFu, cut, o));
    if (lane == 0) s.red_f[warp] = cut;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SW; ++i) cut = fminf(cut, s.red_f[i]);
    if (tid == 0) s.tau = sort_key(cut, V - 1);
  } else {
    cut = mx - kSpan * temp;
    if (tid == 0) s.tau = ~0ull;
  }
  if (mine > -INFINITY && mine >= cut)
    each_word(row, V, rank, CS, [&](int i, float l) {
      if (l >= cut && l > -INFINITY) {
        const int at = atomicAdd(&s.ncand, 1);
        if (at < CAND) s.cand[at] = sort_key(l, i);
        else s.overflow = 1;
      }
    });
  if (tid == 0) s.bmax = mx;
  cluster_sync();

  // ---- the row's largest logit; its total weight where top_k does not bound it
  for (int q = 0; q < CS; ++q) mx = fmaxf(mx, __uint_as_float(peer32(at_rank(&s.bmax, q))));
  r.lmax = mx;
  if (mx == -INFINITY) {  // no word is left
    if (rank == 0 && tid == 0) {
      a.ids[m] = -1;
      if (a.probs) a.probs[m] = 0.0f;
    }
    cluster_sync();
    return;
  }
  auto sum_where = [&](auto take) {  // over the CTA's words
    uint32_t hi = 0;  // a thread has at most 2^11 words (2^20 of a row, 512 threads)
    int lo = 0;
    each_word(row, V, rank, CS, [&](int, float l) {
      int h, g;
      r.parts(l, h, g);
      if (take(l)) { hi += h; lo += g; }
    });
    const unsigned long long t =
        block_sum(s, static_cast<unsigned long long>((static_cast<long long>(hi) << 20) + lo));
    if (tid == 0) s.mass = t;
  };
  auto cluster_mass = [&] {
    unsigned long long t = 0;
    for (int q = 0; q < CS; ++q) t += peer64(at_rank(&s.mass, q));
    return t;
  };
  unsigned long long total = 0;  // of the words kept
  if (k == 0 || k > TOPK_FAST) sum_where([](float l) { return l > -INFINITY; });
  cluster_sync();

  // ---- the cuts and the choice on the listed words, in the first CTA
  if (rank == 0) {
    unsigned long long tau = ~0ull;
    bool good = true;
    for (int q = 0; q < CS; ++q) {
      const unsigned long long t = peer64(at_rank(&s.tau, q));
      tau = t < tau ? t : tau;
      good = good && !peer32(at_rank(&s.overflow, q));
    }
    if (tid == 0) s.nlist = 0;
    __syncthreads();
    for (int q = 0; q < CS; ++q) {
      const int n = min(static_cast<int>(peer32(at_rank(&s.ncand, q))), CAND);
      const uint32_t from = at_rank(s.cand, q);
      for (int i = tid; i < n; i += STH) {
        const unsigned long long cv = peer64(from + 8 * i);
        if (cv <= tau) {
          const int at = atomicAdd(&s.nlist, 1);
          if (at < LIST) s.list[at] = cv;
        }
      }
    }
    __syncthreads();
    const int n = s.nlist;
    good = good && n <= LIST && (k <= TOPK_FAST);
    if (good) {
      const bool complete = tau == ~0ull;  // the list holds every word that weighs anything
      sort_list(s, n);
      Held h = hold(s, r, n);
      if (k > 0) {  // the words past the first k weigh nothing from here on
        good = complete || k <= n;
        unsigned long long t = 0;
#pragma unroll
        for (int i = 0; i < LIST / STH; ++i) {
          if (tid * (LIST / STH) + i >= k) h.w[i] = 0;
          t += h.w[i];
        }
        total = block_sum(s, t);
      } else {
        total = cluster_mass();
      }
      if (good && p < 1.0f) {
        const double want_m = static_cast<double>(p) * static_cast<double>(total);
        unsigned long long x = want_m > 1.0 ? static_cast<unsigned long long>(ceil(want_m)) - 1 : 0;
        if (x >= total) x = total - 1;
        good = pass_at(s, h, 0, x);
        if (good) total = s.found_before + r.units(logit_of(s.found_cv));
      }
      if (good && mp > 0.0f) {
        unsigned long long t = 0;
        int below = 0;  // some listed word is below min_p: the cut is inside the list
#pragma unroll
        for (int i = 0; i < LIST / STH; ++i) {
          if (tid * (LIST / STH) + i >= n) continue;
          const float w = r.weight(logit_of(h.cv[i]));
          if (w >= fminf(mp, 1.0f)) t += h.w[i];
          else below = 1;
        }
        below = __syncthreads_or(below);
        t = block_sum(s, t);
        if (below || complete) total = t < total ? t : total;
        else good = k > 0 || p < 1.0f;  // the cut lies past the list, and past the other cut where there is one
      }
      if (good) {
        const double uw = static_cast<double>(u) * static_cast<double>(total);
        unsigned long long x = uw > 0.0 ? static_cast<unsigned long long>(uw) : 0;
        if (x >= total) x = total - 1;
        good = pass_at(s, h, 0, x);
        if (good && tid == 0) {
          a.ids[m] = static_cast<int>(s.found_cv & ((1u << kIdxBits) - 1));
          if (a.probs)
            a.probs[m] = static_cast<float>(static_cast<double>(r.units(logit_of(s.found_cv))) / static_cast<double>(total));
        }
      }
    }
    if (tid == 0) s.cmd.done = good;
  }
  cluster_sync();
  const bool done = peer32(at_rank(&s.cmd.done, 0)) != 0;
  total = cluster_mass();
  cluster_sync();
  if (done) return;

  // ---- the same cuts over the whole row
  if (k > 0) {
    if (k <= TOPK_FAST) {
      sum_where([](float l) { return l > -INFINITY; });
      cluster_sync();
      total = cluster_mass();
    }
    if (locate(s, row, V, rank, CS, r, static_cast<unsigned long long>(k) - 1, true) && rank == 0)
      total = s.found_before + r.units(logit_of(s.found_cv));
  }
  if (p < 1.0f) {
    const double want_m = static_cast<double>(p) * static_cast<double>(total);
    unsigned long long x = want_m > 1.0 ? static_cast<unsigned long long>(ceil(want_m)) - 1 : 0;
    if (x >= total) x = total - 1;
    locate(s, row, V, rank, CS, r, x, false);
    if (rank == 0) {
      const unsigned long long t = s.found_before + r.units(logit_of(s.found_cv));
      total = t < total ? t : total;
    }
  }
  if (mp > 0.0f) {
    cluster_sync();
    sum_where([&](float l) { return l > -INFINITY && r.weight(l) >= fminf(mp, 1.0f); });
    cluster_sync();
    const unsigned long long t = cluster_mass();
    total = t < total ? t : total;
  }
  const double uw = static_cast<double>(u) * static_cast<double>(total);
  unsigned long long x = uw > 0.0 ? static_cast<unsigned long long>(uw) : 0;
  if (x >= total) x = total - 1;
  locate(s, row, V, rank, CS, r, x, false);
  if (rank == 0 && tid == 0) {
    a.ids[m] = static_cast<int>(s.found_cv & ((1u << kIdxBits) - 1));
    if (a.probs)
      a.probs[m] = static_cast<float>(static_cast<double>(r.units(logit_of(s.found_cv))) / static_cast<double>(total));
  }
  cluster_sync();
}

}  // namespace

size_t sample_workspace_bytes(int64_t, int64_t) { return 256; }

cudaError_t launch_sample(const SampleArgs& a, int bf16, cudaStream_t st) {
  // CTAs per row: as many as fill the device's four CTAs per SM (a row in fewer, larger shares once the rows do), with
  // at least 4096 words each, and at most 2^18, the histograms' room.
  int CS = 1;
  while (CS < 8 && static_cast<int64_t>(a.M) * CS * 2 <= 4 * num_sms() && a.V / (CS * 2) >= 4096) CS *= 2;
  while (CS < 8 && a.V / CS > (1 << 18)) CS *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.M) * CS);
  cfg.blockDim = dim3(STH);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return bf16 ? cudaLaunchKernelEx(&cfg, sample_kernel<__nv_bfloat16>, a, CS)
              : cudaLaunchKernelEx(&cfg, sample_kernel<float>, a, CS);
}

}  // namespace kq
