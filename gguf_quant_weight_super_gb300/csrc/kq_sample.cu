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
//    ones a threshold with about as many words above it as the row needs
//    (top_k of them, else 512 in all).  While the CTAs exchange their largest
//    logits each works out its threshold.
//  * The words above it are listed, in two steps: chunks of 16 bytes that hold
//    one are noted, then every thread looks at a noted one (a warp that lists
//    what few of its lanes found, where they found it, took 27 us in place of 13
//    for top_k = 1000 in one CTA).  A row without top_k sums its total weight in
//    the same second pass (from L2), others only look again at the chunks of the
//    threads whose largest logit is above the threshold.
//  * The first CTA sorts the lists and makes the cuts and the choice on the
//    sorted words.  They are complete above the highest of the CTAs'
//    thresholds, so what falls inside is final.
//  * A row whose cut or token falls outside (flat distributions, large top_k)
//    goes on with a histogram of the whole row: counts and weights in 1024 bins
//    of the distance to the largest logit.  The words of the bin that holds an
//    answer are listed and the word picked among them; where a bin has more
//    words than the list, 1024 bins of the next digits of their sorting key at a
//    time, the index being the last.
// Measured on one GB300, calls in a graph: one row of 151936 (fp32, top-k 20)
// 9.6 us: 1.0 for the first pass, 3.8 for threshold and lists, 1 for fetching
// them, 2.8 for the choice; 16 rows of 262144 (nucleus and min-p) 17.0 us, of
// which 4.5 for the total weight; 256 bf16 rows of mixed settings 66 us: 35 for
// all of them and 28 for the one to four flat ones that are left to the tail.
#include "kq_cache.h"

namespace kq {
namespace {

constexpr int STH = 512;      // threads per CTA
constexpr int SW = STH / 32;
constexpr int CAND = 2048;    // words a CTA lists
constexpr int LIST = 2048;    // words the first CTA works on
constexpr int BINS = 1024;    // two per thread
constexpr int WANT = 512;    // words to list in all for a row without top_k
constexpr int FEW = 64;       // words that one warp decides on
constexpr int TOPK_FAST = 1024;  // top_k up to here by thresholds
constexpr float kSpan = 29.0f;  // exp(-29) < 2^-41: words this far below the largest weigh nothing
constexpr int kIdxBits = 20;

// Which words the cluster looks at next, and what for: from the first CTA to the others.
enum : int { kAll, kDigits, kGather, kNone };
struct Cmd {
  int what;
  int bin;                 // kDigits, kGather: the bin of all words
  int shift;               // kDigits: by the key's 10 bits above shift; kGather: of the key's digits above shift
  unsigned long long pre;  // those digits
};

struct Smem {
  uint32_t count[BINS], limb[2][BINS];
  unsigned long long all_m[BINS];  // the whole row's histogram, in the first CTA
  uint32_t all_c[BINS];
  unsigned long long list[LIST];
  unsigned long long cand[CAND];
  unsigned long long scan_m[SW], red_m[SW];
  int scan_c[SW];
  float red_f[SW];
  unsigned long long mass;      // this CTA's sum
  unsigned long long tau;       // its threshold, as the largest sorting key that is listed for sure
  int ncand, nhit, nlist, listed, done;
  float bmax;
  Cmd cmd;
  unsigned long long found_cv, found_before;  // the word at which a running sum passes, and the sum before it
  int pick, pick_c, pick_n;
  unsigned long long pick_m;
  unsigned long long total, x, base_m;  // whole_row's: the weight kept, what the running sum has to pass, the sum before
  int base_c;
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

// Every word of this CTA's share of the row: chunk(index, 16 bytes) for whole chunks by address, U of them in flight per
// thread (U = 0: none), and word(index, logit) for the up to 14 words outside whole chunks.
template <int U, class X, class FC, class FW>
__device__ __forceinline__ void each_chunk(const X* row, int V, int rank, int CS, FC chunk, FW word) {
  constexpr int E = 16 / static_cast<int>(sizeof(X));
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(X)) % E);
  const int head = off ? min(V, E - off) : 0, chunks = (V - head) / E, tail = V - head - chunks * E;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  const int step = CS * STH;
#pragma unroll 1
  for (int c = rank * STH + static_cast<int>(threadIdx.x); U > 0 && c < chunks; c += U * step) {
    uint4 v[U > 0 ? U : 1];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (c + k * step < chunks) v[k] = __ldg(body + c + k * step);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (c + k * step < chunks) chunk(head + (c + k * step) * E, v[k]);
  }
  if (rank == 0 && static_cast<int>(threadIdx.x) < head + tail) {
    const int t = threadIdx.x, i = t < head ? t : V - 1 - (t - head);
    word(i, one(row + i));
  }
}
// The same, word(index, logit) for all of them, one chunk at a time with the next one in flight: for long bodies, of which
// several copies cost more to fetch than they save.
template <class X, class F>
__device__ __forceinline__ void each_word(const X* row, int V, int rank, int CS, F word) {
  constexpr int E = 16 / static_cast<int>(sizeof(X));
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(X)) % E);
  const int head = off ? min(V, E - off) : 0, chunks = (V - head) / E, step = CS * STH;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  int c = rank * STH + static_cast<int>(threadIdx.x);
  uint4 next;
  if (c < chunks) next = __ldg(body + c);
#pragma unroll 1
  for (; c < chunks; c += step) {
    const uint4 v = next;
    if (c + step < chunks) next = __ldg(body + c + step);
    each4(row, v, head + c * E, word);
  }
  each_chunk<0>(row, V, rank, CS, [](int, uint4) {}, word);
}
__device__ __forceinline__ float largest(const float*, uint4 v) {
  return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}
__device__ __forceinline__ float largest(const __nv_bfloat16*, uint4 v) {  // NaN counts for nothing
  auto pair = [](uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); };
  const __nv_bfloat162 x = __hmax2(__hmax2(pair(v.x), pair(v.y)), __hmax2(pair(v.z), pair(v.w)));
  return fmaxf(__low2float(x), __high2float(x));
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
  float zs;       // bins per unit of logit: kSpan over all of them, whatever the temperature
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
  // the distance to the largest logit in bins
  __device__ __forceinline__ float depth(float l) const { return l == lmax ? 0.0f : fminf((lmax - l) * zs, BINS - 1.0f); }
  __device__ __forceinline__ int bin(float l) const { return static_cast<int>(depth(l)); }
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
#pragma unroll
  for (int w = 0; w < SW - 1; ++w)
    if (w < warp) { im += s.scan_m[w]; ic += s.scan_c[w]; }
  m = im;
  c = ic;
}
// Sorts s.list[0, n) ascending, n <= LIST.  Up to 320 words: each counts those before it.  More: the words'
// depths, stretched over the bins, nearly sort them (a few words per bin), and inside a bin each word counts those before
// it.  Where a bin holds many (equal logits): bitonic, a warp's 32 threads comparing within the same 64 places while the
// stride is 32 or less, so that only wider steps need the whole block's barrier.  Takes s.cand and s.count as scratch.
__device__ __noinline__ void sort_list(Smem& s, const Row r, int n) {
  constexpr int PER = LIST / STH, MANY = 160, MOST = 320;
  if (n <= MOST) {
    const int t = threadIdx.x;
    const unsigned long long mine = t < n ? s.list[t] : 0;
    int place = 0;
    if (t < n) {
#pragma unroll 4
      for (int j = 0; j < n; ++j) place += s.list[j] < mine;
    }
    __syncthreads();
    if (t < n) s.list[place] = mine;
    __syncthreads();
    return;
  }
  unsigned long long cv[PER];
  float z[PER], deepest = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = static_cast<int>(threadIdx.x) + i * STH;
    cv[i] = j < n ? s.list[j] : ~0ull;
    z[i] = j < n ? r.depth(logit_of(cv[i])) : 0.0f;
    deepest = fmaxf(deepest, z[i]);
  }
  deepest = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(deepest)));  // not negative
  if ((threadIdx.x & 31) == 0) s.red_f[threadIdx.x >> 5] = deepest;
  s.count[2 * threadIdx.x] = s.count[2 * threadIdx.x + 1] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SW; ++i) deepest = fmaxf(deepest, s.red_f[i]);
  const float f = deepest > 0.0f ? (BINS - 1) / deepest : 0.0f;
  int at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (cv[i] != ~0ull) at[i] = atomicAdd(&s.count[static_cast<int>(fminf(z[i] * f, BINS - 1.0f))], 1);
  __syncthreads();
  const int c0 = s.count[2 * threadIdx.x], c1 = s.count[2 * threadIdx.x + 1];
  if (!__syncthreads_or(max(c0, c1) > MANY)) {
    unsigned long long none = 0;
    int before = c0 + c1;
    block_scan(s, none, before);
    s.count[2 * threadIdx.x] = before;
    s.count[2 * threadIdx.x + 1] = before + c0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (cv[i] != ~0ull) s.cand[s.count[static_cast<int>(fminf(z[i] * f, BINS - 1.0f))] + at[i]] = cv[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (cv[i] == ~0ull) continue;
      const int b = static_cast<int>(fminf(z[i] * f, BINS - 1.0f));
      const int from = s.count[b], to = b + 1 < BINS ? s.count[b + 1] : n;
      int place = from;
      for (int j = from; j < to; ++j) place += s.cand[j] < cv[i];
      s.list[place] = cv[i];
    }
    __syncthreads();
    return;
  }
  int size = 64;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += STH) s.list[i] = ~0ull;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < size / 2; t += STH) {
        const int i = 2 * t - (t & (j - 1)), x = i + j;  // i has bit j clear
        const unsigned long long a = s.list[i], b = s.list[x];
        if ((a > b) == ((i & k) == 0)) { s.list[i] = b; s.list[x] = a; }
      }
      if (j > 32) __syncthreads();
      else __syncwarp();
    }
    if (k >= 64) __syncthreads();  // the next step is a wide one
  }
  __syncthreads();
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
__device__ __forceinline__ void peer_store32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int peer_add(uint32_t addr, int v) {
  int r;
  asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(r) : "r"(addr), "r"(v) : "memory");
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The four words of the sorted list that thread t holds, and the weight before them.
struct Held {
  unsigned long long w[LIST / STH], before;
};
__device__ __forceinline__ Held hold(Smem& s, const Row& r, int n) {
  Held h;
  h.before = 0;
  int c = 0;
#pragma unroll
  for (int i = 0; i < LIST / STH; ++i) {
    const int j = static_cast<int>(threadIdx.x) * (LIST / STH) + i;
    h.w[i] = j < n ? r.units(logit_of(s.list[j])) : 0;
    h.before += h.w[i];
  }
  block_scan(s, h.before, c);
  return h;
}
// The held word at which the running sum, from base on, passes x (by_count: the x-th of the list): found_cv, found_before;
// false where there is none.
__device__ __forceinline__ bool pass_at(Smem& s, const Held& h, unsigned long long base, unsigned long long x, bool by_count) {
  __syncthreads();
  if (threadIdx.x == 0) s.pick = -1;
  __syncthreads();
  unsigned long long c = base + h.before;
#pragma unroll
  for (int i = 0; i < LIST / STH; ++i) {
    const int j = static_cast<int>(threadIdx.x) * (LIST / STH) + i;
    if (by_count ? static_cast<unsigned long long>(j) == x && h.w[i] > 0 : c <= x && x < c + h.w[i]) {
      s.found_cv = s.list[j];
      s.found_before = c;
      s.pick = j;
    }
    c += h.w[i];
  }
  __syncthreads();
  return s.pick >= 0;
}

// The running sums that the last kept word passes for top_p (kept: the words with less than p * total before them) and
// that the token passes for u, as integers: f * total exactly, f being a 64-bit fraction.
__device__ __forceinline__ unsigned long long fraction(float f) {  // 0 <= f < 1
  const uint32_t b = __float_as_uint(f);
  const int sh = static_cast<int>(b >> 23) - 86;
  const unsigned long long man = (b & 0x7FFFFFu) | 0x800000u;
  return sh >= 0 ? man << sh : sh > -24 ? man >> -sh : 0;
}
__device__ __forceinline__ unsigned long long nucleus(float p, unsigned long long total) {
  if (!(p > 0.0f)) return 0;
  const unsigned long long f = fraction(p), hi = __umul64hi(f, total);
  return f * total != 0 || hi == 0 ? hi : hi - 1;
}
__device__ __forceinline__ unsigned long long share(float u, unsigned long long total) {
  if (!(u > 0.0f)) return 0;
  return u < 1.0f ? __umul64hi(fraction(u), total) : total - 1;
}
__device__ __forceinline__ void write_row(const SampleArgs& a, int m, const Row& r, unsigned long long cv,
                                          unsigned long long total) {
  a.ids[m] = static_cast<int>(cv & ((1u << kIdxBits) - 1));
  if (a.probs) a.probs[m] = __ull2float_rn(r.units(logit_of(cv))) / __ull2float_rn(total);
}

// A place in a list for each lane that is `on` (every lane of the warp calls it).
__device__ __forceinline__ int push_at(int* counter, bool on) {
  const uint32_t who = __ballot_sync(0xFFFFFFFFu, on);
  const int lane = threadIdx.x & 31;
  int base = 0;
  if (lane == 0 && who) base = atomicAdd(counter, __popc(who));
  return __shfl_sync(0xFFFFFFFFu, base, 0) + __popc(who & ((1u << lane) - 1u));
}

// The cuts and the choice on n <= FEW listed words, by one warp, two words per lane.  total: the row's weight where k is 0.
// Returns whether the answer lies in the list; then the word in cv_out and the kept weight in total.  Runs once per row:
// loops stay rolled, since what it costs is fetching its code.
__device__ __noinline__ bool choose_in_warp(const unsigned long long* list, bool sorted, const Row r, int n, bool complete, int k,
                                            float p, float mp, float u, unsigned long long& total, unsigned long long& cv_out) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31;
  unsigned long long v0 = lane < n ? list[lane] : ~0ull, v1 = lane + 32 < n ? list[lane + 32] : ~0ull;
  if (!sorted) {  // bitonic over places lane and lane + 32
#pragma unroll 1
    for (int k2 = 2; k2 <= 32; k2 <<= 1)
#pragma unroll 1
      for (int j = k2 >> 1; j > 0; j >>= 1) {
        const unsigned long long o0 = __shfl_xor_sync(kAll, v0, j), o1 = __shfl_xor_sync(kAll, v1, j);
        const bool least = ((lane & j) == 0) == ((lane & k2) == 0);  // k2 = 32: the lower half ascends, the upper descends
        v0 = (v0 < o0) == least ? v0 : o0;
        v1 = (v1 < o1) == (k2 == 32 ? (lane & j) != 0 : least) ? v1 : o1;
      }
    if (v0 > v1) { const unsigned long long x = v0; v0 = v1; v1 = x; }
#pragma unroll 1
    for (int j = 16; j > 0; j >>= 1) {
      const unsigned long long o0 = __shfl_xor_sync(kAll, v0, j), o1 = __shfl_xor_sync(kAll, v1, j);
      const bool least = (lane & j) == 0;
      v0 = (v0 < o0) == least ? v0 : o0;
      v1 = (v1 < o1) == least ? v1 : o1;
    }
  }
  const unsigned long long w0 = lane < n ? r.units(logit_of(v0)) : 0, w1 = lane + 32 < n ? r.units(logit_of(v1)) : 0;
  unsigned long long c0 = w0, c1 = w1;  // running sums with the word
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long t0 = __shfl_up_sync(kAll, c0, o), t1 = __shfl_up_sync(kAll, c1, o);
    if (lane >= o) { c0 += t0; c1 += t1; }
  }
  c1 += __shfl_sync(kAll, c0, 31);
  const unsigned long long sum = __shfl_sync(kAll, c1, 31);
  // the place of the word at which the running sum passes x, 64: none
  auto pass = [&](unsigned long long x) {
    const uint32_t a = __ballot_sync(kAll, x < c0), b = __ballot_sync(kAll, x < c1);
    return a ? __ffs(a) - 1 : b ? 31 + __ffs(b) : 64;
  };
  auto with = [&](int at) { return __shfl_sync(kAll, at < 32 ? c0 : c1, at & 31); };
  if (k > 0) {
    if (k > n && !complete) return false;
    total = k >= n ? sum : with(k - 1);
  }
  bool bounded = k > 0;  // the kept words end inside the list
  if (p < 1.0f) {
    const int at = pass(nucleus(p, total));
    if (at < 64) {
      total = min(total, with(at));
      bounded = true;
    }
  }
  if (mp > 0.0f) {
    const float least = fminf(mp, 1.0f);
    const int in = __popc(__ballot_sync(kAll, lane < n && r.weight(logit_of(v0)) >= least)) +
                   __popc(__ballot_sync(kAll, lane + 32 < n && r.weight(logit_of(v1)) >= least));
    if (in < n || complete) {
      total = min(total, with(max(in, 1) - 1));
      bounded = true;
    }
  }
  // a nucleus that ends past the list is only harmless if another cut ends inside, and no cut at all only for u inside
  if (!bounded && (p < 1.0f || mp > 0.0f)) return false;
  const int at = pass(share(u, total));
  if (at >= 64) return false;
  cv_out = __shfl_sync(kAll, at < 32 ? v0 : v1, at & 31);
  return true;
}

// This CTA's sum of the weights that `take` takes, into s.mass.  also(index, chunk): what else is done with each chunk.
template <class X, class F, class G>
__device__ __forceinline__ void sum_where(Smem& s, const X* row, int V, int rank, int CS, const Row& r, F take, G also) {
  uint32_t hi = 0;  // a thread has at most 2^11 words (2^20 of a row, 512 threads)
  int lo = 0;
  auto word = [&](int i, float l) {
    int h, g;
    r.parts(l, h, g);
    if (take(i, l)) { hi += h; lo += g; }
  };
  each_chunk<4>(
      row, V, rank, CS,
      [&](int i, uint4 v) {
        also(i, v);
        each4(row, v, i, word);
      },
      word);
  const unsigned long long t = block_sum(s, static_cast<unsigned long long>((static_cast<long long>(hi) << 20) + lo));
  if (threadIdx.x == 0) s.mass = t;
}
// The same for all words, two at a time: half the instructions, which bound it where a CTA has a whole row.  The largest
// logit and the scale are finite.
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
  return a;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
  return a;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return a;
}
template <class F>
__device__ __forceinline__ void each_pair(const float*, uint4 v, F f) {
  f(__uint_as_float(v.x), __uint_as_float(v.y)), f(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <class F>
__device__ __forceinline__ void each_pair(const __nv_bfloat16*, uint4 v, F f) {
  f(bf16_lo(v.x), bf16_hi(v.x)), f(bf16_lo(v.y), bf16_hi(v.y)), f(bf16_lo(v.z), bf16_hi(v.z)), f(bf16_lo(v.w), bf16_hi(v.w));
}
template <class X, class G>
__device__ __forceinline__ void sum_all(Smem& s, const X* row, int V, int rank, int CS, const Row& r, G also) {
  uint32_t hi = 0, lo = 0, pairs = 0;
  const F2 less(-r.lmax), c(r.c), unit(1048576.0f), magic(12582912.0f), minus(-1.0f);
  each_chunk<sizeof(X)>(
      row, V, rank, CS,
      [&](int i, uint4 v) {
        also(i, v);
        each_pair(row, v, [&](float a, float b) {
          ((F2(a, b) + less) * c).get(a, b);
          const F2 w(fmaxf(ex2(a), 0.0f), fmaxf(ex2(b), 0.0f));  // a NaN weighs nothing
          const F2 h = fma2(w, unit, magic), l = fma2(fma2(w, unit, fma2(h, minus, magic)), unit, magic);
          h.get(a, b);
          hi += __float_as_uint(a) + __float_as_uint(b);
          l.get(a, b);
          lo += __float_as_uint(a) + __float_as_uint(b);
          ++pairs;
        });
      },
      [&](int, float l) {
        int h, g;
        r.parts(l, h, g);
        if (l > -INFINITY) { hi += h; lo += g; }
      });
  hi -= pairs * 0x96800000u;
  lo -= pairs * 0x96800000u;
  const unsigned long long t =
      block_sum(s, static_cast<unsigned long long>((static_cast<long long>(hi) << 20) + static_cast<int>(lo)));
  if (threadIdx.x == 0) s.mass = t;
}
// Lists the words of a chunk from `cut` up.
template <class X>
__device__ __noinline__ void list_chunk(Smem& s, const X* row, int i, uint4 v, float cut) {
  int n = 0;
  each4(row, v, i, [&](int, float l) { n += l >= cut && l > -INFINITY; });
  if (n == 0) return;
  int at = atomicAdd(&s.ncand, n);
  each4(row, v, i, [&](int j, float l) {
    if (l >= cut && l > -INFINITY) {
      if (at < CAND) s.cand[at] = sort_key(l, j);
      ++at;
    }
  });
}

__device__ __forceinline__ unsigned long long cluster_mass(Smem& s, int CS) {
  unsigned long long t = 0;
  for (int q = 0; q < CS; ++q) t += peer64(at_rank(&s.mass, q));
  return t;
}

// ---- the whole-row path

// A histogram's two bins of this thread, and what lies before them.
struct Bins {
  unsigned long long m[2], pm;
  int c[2], pc;
};
// A bin's weight in two words; the higher one is added to where the lower one passes 2^32 or the weight does, which is
// seldom in the rows that come here.
__device__ __forceinline__ void add_weight(Smem& s, int d, unsigned long long w) {
  const uint32_t lo = static_cast<uint32_t>(w), before = atomicAdd(&s.limb[0][d], lo);
  const uint32_t hi = static_cast<uint32_t>(w >> 32) + (before + lo < before);
  if (hi) atomicAdd(&s.limb[1][d], hi);
}
// The sum of the cluster's histograms, into the first CTA's `to` (weights) and `to_n` (words).  Each CTA sums its share of
// the bins: one that read all of them from the others (128 KB) took 8 us.
__device__ __forceinline__ void share_bins(Smem& s, unsigned long long* to, uint32_t* to_n, int rank, int CS) {
  const int share = BINS / CS, each = max(1, CS / 2);  // CTAs are read by `each` groups of threads
  for (int i = threadIdx.x; i < share * each; i += STH) {
    const int b = rank * share + i % share;
    unsigned long long m = 0, c = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int q = i / share * 2 + k;
      if (q < CS) {
        c += peer32(at_rank(&s.count[b], q));
        m += peer32(at_rank(&s.limb[0][b], q)) + (static_cast<unsigned long long>(peer32(at_rank(&s.limb[1][b], q))) << 32);
      }
    }
    s.cand[i] = m;
    s.cand[BINS + i] = c;
  }
  __syncthreads();
  const uint32_t to_m = at_rank(to, 0), to_c = at_rank(to_n, 0);
  for (int i = threadIdx.x; i < share; i += STH) {
    unsigned long long m = 0, c = 0;
    for (int k = 0; k < each; ++k) {
      m += s.cand[k * share + i];
      c += s.cand[BINS + k * share + i];
    }
    peer_store64(to_m + 8 * (rank * share + i), m);
    peer_store32(to_c + 4 * (rank * share + i), static_cast<uint32_t>(c));
  }
}
__device__ __forceinline__ Bins read_bins(Smem& s, const unsigned long long* m, const uint32_t* c) {
  Bins h;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    h.m[e] = m[2 * threadIdx.x + e];
    h.c[e] = static_cast<int>(c[2 * threadIdx.x + e]);
  }
  h.pm = h.m[0] + h.m[1];
  h.pc = h.c[0] + h.c[1];
  block_scan(s, h.pm, h.pc);
  return h;
}
// The bin in which the running sum of weights (by_count: of words), from base on, passes x: s.pick (-1: none), s.pick_m
// and s.pick_c before it, s.pick_n words in it.
__device__ __forceinline__ void pick_bin(Smem& s, const Bins& h, unsigned long long base_m, int base_c,
                                         unsigned long long x, bool by_count) {
  __syncthreads();
  if (threadIdx.x == 0) s.pick = -1;
  __syncthreads();
  unsigned long long m = base_m + h.pm;
  int c = base_c + h.pc;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const unsigned long long before = by_count ? c : m, in = by_count ? h.c[e] : h.m[e];
    if (before <= x && x < before + in) {
      s.pick = 2 * threadIdx.x + e;
      s.pick_m = m;
      s.pick_c = c;
      s.pick_n = h.c[e];
    }
    m += h.m[e];
    c += h.c[e];
  }
  __syncthreads();
}
// The word of s.list[0, n), in any order, at which the running sum, from base on, passes x, as by pick_bin: found_cv and
// found_before.  The range of the keys that are left is cut into 1024 bins and one of them picked, until at most 32 words
// are left for one warp.  The keys of bf16 logits are taken without the 16 bits that all have alike, and those of indices
// without the bits above V's: the list has few different logits then, and bins by logit alone would hold hundreds of words,
// whose additions wait for one another (9 us in place of 4 for 2048 words).
template <class X>
__device__ __forceinline__ void pass_in_list(Smem& s, const Row r, int V, int n, unsigned long long base_m, int base_c,
                                          unsigned long long x, bool by_count) {
  constexpr int PER = LIST / STH, kSame = sizeof(X) == 2 ? 16 : 0;
  const int bits = 32 - __clz(V);
  auto place = [&](unsigned long long cv) {
    return (cv >> (kIdxBits + kSame) << bits) | (cv & ((1u << kIdxBits) - 1));
  };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long at[PER], w[PER];  // ~0: not among those left
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = static_cast<int>(threadIdx.x) + i * STH;
    at[i] = j < n ? place(s.list[j]) : ~0ull;
    w[i] = j < n ? r.units(logit_of(s.list[j])) : 0;
  }
  while (n > 32) {
    unsigned long long least = ~0ull, most = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      least = min(least, at[i]);
      if (at[i] != ~0ull) most = max(most, at[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
      most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    }
    if (lane == 0) { s.red_m[warp] = least; s.scan_m[warp] = most; }
    for (int i = threadIdx.x; i < BINS; i += STH) { s.count[i] = 0; s.limb[0][i] = 0; s.limb[1][i] = 0; }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SW; ++i) { least = min(least, s.red_m[i]); most = max(most, s.scan_m[i]); }
    const int shift = max(0, 54 - __clzll(static_cast<long long>(most - least)));  // most - least in 1024 steps
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at[i] != ~0ull) {
        const int d = static_cast<int>((at[i] - least) >> shift);
        atomicAdd(&s.count[d], 1u);
        atomicAdd(&s.limb[0][d], static_cast<uint32_t>(w[i]) & 0xFFFFFu);  // at most 2048 of them: below 2^31
        atomicAdd(&s.limb[1][d], static_cast<uint32_t>(w[i] >> 20));
      }
    __syncthreads();
    Bins h;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int b = 2 * threadIdx.x + e;
      h.c[e] = s.count[b];
      h.m[e] = (static_cast<unsigned long long>(s.limb[1][b]) << 20) + s.limb[0][b];
    }
    h.pm = h.m[0] + h.m[1];
    h.pc = h.c[0] + h.c[1];
    block_scan(s, h.pm, h.pc);
    pick_bin(s, h, base_m, base_c, x, by_count);
    const int pick = s.pick;
    if (pick < 0) return;  // none
    base_m = s.pick_m;
    base_c = s.pick_c;
    n = s.pick_n;  // each bin is narrower than all of them by 2^10: six rounds at most
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at[i] != ~0ull && static_cast<int>((at[i] - least) >> shift) != pick) at[i] = ~0ull;
    __syncthreads();
  }
  if (threadIdx.x == 0) s.pick_n = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (at[i] != ~0ull) s.cand[atomicAdd(&s.pick_n, 1)] = s.list[static_cast<int>(threadIdx.x) + i * STH];
  __syncthreads();
  if (warp == 0) {
    const unsigned long long mine = lane < n ? s.cand[lane] : ~0ull, has = lane < n ? r.units(logit_of(mine)) : 0;
    unsigned long long before = base_m, count = base_c;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const unsigned long long o = __shfl_sync(0xFFFFFFFFu, mine, i), ow = __shfl_sync(0xFFFFFFFFu, has, i);
      if (o < mine) { before += ow; ++count; }
    }
    if (lane < n && (by_count ? count == x : before <= x && x < before + has)) {
      s.found_cv = mine;
      s.found_before = before;
    }
  }
  __syncthreads();
}
// A row's settings: temperature not above 0 is the first word; k = 0: no top_k.
__device__ __forceinline__ void settings(const SampleArgs& a, int m, float& temp, int& k, float& p, float& mp, float& u) {
  temp = a.temperature ? __ldg(a.temperature + m) : 1.0f;
  k = a.top_k ? __ldg(a.top_k + m) : 0;
  p = a.top_p ? __ldg(a.top_p + m) : 1.0f;
  mp = a.min_p ? __ldg(a.min_p + m) : 0.0f;
  u = __ldg(a.u + m);
  if (!(temp > 0.0f)) {
    temp = 1.0f;
    k = 1;
  }
  if (k < 0 || k >= a.V) k = 0;
}

// The weight of the words down to the one with the key `last` that weigh at least `least`, every CTA of the cluster.
template <class X>
__device__ __noinline__ void sum_cut(Smem& s, const X* row, int V, int rank, int CS, const Row r, unsigned long long last,
                                     float least) {
  sum_where(
      s, row, V, rank, CS, r,
      [&](int i, float l) { return l > -INFINITY && sort_key(l, i) <= last && r.weight(l) >= least; }, [](int, uint4) {});
}

// The cuts and the choice over the whole row, every CTA of the cluster.  total: the row's weight, 0 if it is not known.
// Up to three words are looked for, one after the other: the top_k-th, the last of the nucleus, the token.  Each is found
// as the word at which the running sum of weights (for the top_k-th: of words that weigh anything) passes x: first its bin
// in the histogram of the whole row, which is made once, then among the words of that bin.  What is kept across the
// cluster's barriers is in registers or shared memory: each of them empties the cache that local memory is read through.
template <class X>
__device__ __noinline__ void whole_row(Smem& s, const SampleArgs& a, const X* row, int m, int rank, int CS, const Row r_in,
                                       unsigned long long total) {
  const Row r = r_in;  // a copy that no store can change
  enum : int { kCount, kNucleus, kToken };
  const int V = a.V;
  auto cut_total = [&](unsigned long long last, float least) {
    sum_cut(s, row, V, rank, CS, r, last, least);
    cluster_sync();
    const unsigned long long t = cluster_mass(s, CS);
    cluster_sync();
    return t;
  };
  if (total == 0) total = cut_total(~0ull, 0.0f);
  if (threadIdx.x == 0) s.total = total;
  bool have = false;  // the histogram of the whole row
  int step = -1;      // the one before
#pragma unroll 1
  do {
    {
      float temp, p, mp, u;
      int k;
      settings(a, m, temp, k, p, mp, u);
      step = step < kCount && k > 0 ? kCount : step < kNucleus && p < 1.0f ? kNucleus : kToken;
      unsigned long long t = ~0ull;
      if (step == kToken && mp > 0.0f) t = cut_total(~0ull, fminf(mp, 1.0f));
      if (threadIdx.x == 0) {
        t = min(t, s.total);
        s.total = t;
        s.x = step == kCount ? static_cast<unsigned long long>(k) - 1 : step == kNucleus ? nucleus(p, t) : share(u, t);
        s.base_m = 0;
        s.base_c = 0;
      }
      __syncthreads();
    }
    const bool by_count = step == kCount;
    unsigned long long pre = 0;
    int what = kAll, shift = 0, bin = 0;
    auto sums = [&] { return what == kAll ? s.all_m : s.list; };  // of digits: where nothing is listed yet
    auto counts = [&] { return what == kAll ? s.all_c : reinterpret_cast<uint32_t*>(s.list + BINS); };
#pragma unroll 1
    for (;;) {
      if (have) {
        if (rank == 0) {
          pick_bin(s, read_bins(s, sums(), counts()), s.base_m, s.base_c, s.x, by_count);
          if (threadIdx.x == 0) {
            if (s.pick >= 0) { s.base_m = s.pick_m; s.base_c = s.pick_c; }
            const bool fits = s.pick_n <= LIST;
            if (what == kAll) {
              s.cmd.bin = s.pick;
              s.cmd.shift = fits ? 64 : 42;
            } else {
              s.cmd.pre = (shift + 10 < 52 ? pre >> (shift + 10) << (shift + 10) : 0) | (static_cast<unsigned long long>(s.pick) << shift);
              s.cmd.shift = fits ? shift : shift - 10;
            }
            s.cmd.what = s.pick < 0 ? kNone : fits ? kGather : kDigits;
            s.nlist = 0;
          }
        }
        if (threadIdx.x == 0) s.ncand = 0;
        cluster_sync();  // the command is written, and the first CTA's list is empty
        what = static_cast<int>(peer32(at_rank(&s.cmd.what, 0)));
        bin = static_cast<int>(peer32(at_rank(&s.cmd.bin, 0)));
        shift = static_cast<int>(peer32(at_rank(&s.cmd.shift, 0)));
        pre = peer64(at_rank(&s.cmd.pre, 0));
        if (what == kNone) {
          cluster_sync();  // every CTA has read the command
          break;
        }
      }
      if (what != kGather) {
        for (int i = threadIdx.x; i < BINS; i += STH) { s.count[i] = 0; s.limb[0][i] = 0; s.limb[1][i] = 0; }
        __syncthreads();
      }
      if (what == kAll) {
        each_word(row, V, rank, CS, [&](int, float l) {
          const unsigned long long w = r.units(l);
          if (!(l > -INFINITY) || w == 0) return;
          const int d = r.bin(l);
          atomicAdd(&s.count[d], 1u);
          add_weight(s, d, w);
        });
      } else {
        each_word(row, V, rank, CS, [&](int i, float l) {
          if (!(l > -INFINITY) || r.bin(l) != bin) return;
          const unsigned long long cv = sort_key(l, i), w = r.units(l);
          if (w == 0) return;
          if (what == kGather) {
            if (shift < 64 && (cv >> shift) != (pre >> shift)) return;
            s.cand[min(atomicAdd(&s.ncand, 1), CAND - 1)] = cv;  // at most LIST of all the CTAs
          } else {
            if (shift + 10 < 52 && (cv >> (shift + 10)) != (pre >> (shift + 10))) return;
            const int d = static_cast<int>(cv >> shift) & (BINS - 1);
            atomicAdd(&s.count[d], 1u);
            add_weight(s, d, w);
          }
        });
      }
      if (what == kGather) {
        __syncthreads();
        const int n = min(s.ncand, CAND);
        if (threadIdx.x == 0) s.listed = peer_add(at_rank(&s.nlist, 0), n);
        __syncthreads();
        const uint32_t to = at_rank(s.list, 0);
        for (int i = threadIdx.x; i < n; i += STH)
          if (s.listed + i < LIST) peer_store64(to + 8 * (s.listed + i), s.cand[i]);
        cluster_sync();
        if (rank == 0) pass_in_list<X>(s, r, V, min(s.nlist, LIST), s.base_m, s.base_c, s.x, by_count);
        break;
      }
      cluster_sync();
      share_bins(s, sums(), counts(), rank, CS);
      cluster_sync();
      have = true;
    }
    if (by_count) {
      cluster_sync();
      const unsigned long long kth = peer64(at_rank(&s.found_cv, 0));
      cluster_sync();
      if (what != kNone) {  // else fewer words weigh anything
        const unsigned long long t = cut_total(kth, 0.0f);
        if (threadIdx.x == 0) s.total = t;
      }
    } else if (step == kNucleus && rank == 0 && threadIdx.x == 0) {
      s.total = min(s.total, s.found_before + r.units(logit_of(s.found_cv)));
    }
  } while (step != kToken);
  if (rank == 0 && threadIdx.x == 0) write_row(a, m, r, s.found_cv, s.total);
}

__device__ __forceinline__ Row row_of(float lmax, float temp) {
  Row r;
  r.lmax = lmax;
  r.c = 1.4426950408889634f / temp;
  r.zs = static_cast<float>(BINS) / kSpan / temp;
  return r;
}

// Rows left to the tail kernel: count, CTAs that have left it, and the rows (null: none are left).
struct Left {
  int m;
  float lmax;
  unsigned long long total;  // the row's weight; 0: not known yet
};
struct Tail {
  int *count, *left;
  Left* rows;
};

template <class X>
__global__ void __launch_bounds__(STH, 2) sample_kernel(const __grid_constant__ SampleArgs a, int CS, Tail tail) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = blockIdx.x / CS, rank = blockIdx.x - m * CS, V = a.V;
  const X* row = static_cast<const X*>(a.logits) + m * a.row_stride;
  float temp, p, mp, u;
  int k;
  settings(a, m, temp, k, p, mp, u);

  // ---- each thread's largest logit, and the CTA's
  for (int i = tid; i < BINS; i += STH) s.count[i] = 0;
  float mine = -INFINITY;
  each_chunk<8>(
      row, V, rank, CS, [&](int, uint4 v) { mine = fmaxf(mine, largest(row, v)); },
      [&](int, float l) { mine = fmaxf(mine, l); });
  float mx = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) s.red_f[warp] = mx;
  if (tid == 0) { s.ncand = 0; s.nhit = 0; s.nlist = 0; s.done = 0; s.pick = BINS; }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SW; ++i) mx = fmaxf(mx, s.red_f[i]);
  if (tid == 0) s.bmax = mx;
  cluster_arrive();

  // ---- meanwhile the threshold: the smallest of the threads' largest logits in the first bins that hold enough of them
  const bool by_top_k = k > 0 && k <= TOPK_FAST;
  Row r = row_of(mx, temp);
  // with n words above the threshold spread over the threads at random, 1 - exp(-n / threads) of them have one
  const float per = static_cast<float>(by_top_k ? k + k / 4 + 32 : WANT) / static_cast<float>(CS);
  // (the CTA with the highest threshold has at least `want` words above it: small top_k are met for certain)
  const int want = max(by_top_k ? min(k, 128) : 8, static_cast<int>(STH * (1.0f - __expf(-fminf(per, 1200.0f) / STH))));
  const bool some = mine > -INFINITY && (mine == mx || (mx - mine) * r.zs < static_cast<float>(BINS));
  const int bin = some ? r.bin(mine) : BINS;
  if (some) atomicAdd(&s.count[bin], 1u);
  __syncthreads();
  {
    unsigned long long none = 0;
    const int c0 = s.count[2 * tid], c1 = s.count[2 * tid + 1];
    int before = c0 + c1;
    block_scan(s, none, before);
    if (before < want && before + c0 >= want) s.pick = 2 * tid;
    else if (before + c0 < want && before + c0 + c1 >= want) s.pick = 2 * tid + 1;
  }
  __syncthreads();
  const int last = s.pick;  // BINS: there are not enough; then all that weighs anything is listed
  float cut = some && bin <= last ? mine : INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) cut = fminf(cut, __shfl_xor_sync(0xFFFFFFFFu, cut, o));
  if (lane == 0) s.red_f[warp] = cut;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SW; ++i) cut = fminf(cut, s.red_f[i]);
  if (last == BINS) cut = mx - kSpan * temp;
  if (tid == 0) s.tau = last == BINS ? ~0ull : sort_key(cut, V - 1);
  cluster_wait();
  {
    const float other = lane < CS ? __uint_as_float(peer32(at_rank(&s.bmax, lane))) : -INFINITY;
    mx = fmaxf(mx, other);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    mx = __shfl_sync(0xFFFFFFFFu, mx, 0);
  }
  r.lmax = mx;

  // ---- the words above the threshold; the row's total weight where top_k does not bound it
  // Chunks with a word above it are noted, then all threads look at the noted ones: a warp would go through its few hits
  // one by one where it found them.
  int* hits = reinterpret_cast<int*>(s.list);
  constexpr int HITS = 2 * LIST;
  auto hit = [&](int i, uint4 v) {
    const float x = largest(row, v);
    if (x >= cut && x > -INFINITY) {
      const int at = atomicAdd(&s.nhit, 1);
      if (at < HITS) hits[at] = i;
    }
  };
  if (by_top_k) {
    // the chunks of the threads whose largest logit is above the threshold, shared out over all threads: a few loads each,
    // where those threads alone would go through all of theirs again
    const bool on = mine >= cut && mine > -INFINITY;
    const int at = push_at(&s.nlist, on);
    if (on) s.count[at] = tid;
    __syncthreads();
    constexpr int E = 16 / static_cast<int>(sizeof(X)), U = 4;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(X)) % E), head = off ? min(V, E - off) : 0;
    const int chunks = (V - head) / E, step = CS * STH, n = max(s.nlist, 1), groups = STH / n, group = tid / n;
    const uint4* body = reinterpret_cast<const uint4*>(row + head);
    // thread h of a group takes every groups-th chunk of the h-th of those threads
    const int from = rank * STH + static_cast<int>(s.count[tid - group * n]);
#pragma unroll 1
    for (int c = from + group * step; group < groups && s.nlist > 0 && c < chunks; c += U * groups * step) {
      uint4 v[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + i * groups * step < chunks) v[i] = __ldg(body + c + i * groups * step);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + i * groups * step < chunks) hit(head + (c + i * groups * step) * E, v[i]);
    }
  } else if (mx < INFINITY && r.c < INFINITY) {
    sum_all(s, row, V, rank, CS, r, hit);
  } else {
    sum_where(s, row, V, rank, CS, r, [&](int, float l) { return l > -INFINITY; }, hit);
  }
  __syncthreads();
  const int nh = s.nhit;
  for (int i = tid; i < min(nh, HITS); i += STH)
    list_chunk(s, row, hits[i], __ldg(reinterpret_cast<const uint4*>(row + hits[i])), cut);
  if (nh > HITS && tid == 0) atomicAdd(&s.ncand, CAND + 1);  // too many
  each_chunk<0>(row, V, rank, CS, [](int, uint4) {}, [&](int i, float l) {
    if (l >= cut && l > -INFINITY) {
      const int at = atomicAdd(&s.ncand, 1);
      if (at < CAND) s.cand[at] = sort_key(l, i);
    }
  });
  cluster_sync();

  // ---- the cuts and the choice on the listed words, in the first CTA
  unsigned long long sum = 0;  // the row's weight, where it is known
  if (rank == 0) {
    if (tid == 0) s.nlist = 0;
    unsigned long long tau = lane < CS ? peer64(at_rank(&s.tau, lane)) : ~0ull;
    const int listed = lane < CS ? static_cast<int>(peer32(at_rank(&s.ncand, lane))) : 0;
    if (lane < CS && !by_top_k) sum = peer64(at_rank(&s.mass, lane));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      tau = min(tau, __shfl_xor_sync(0xFFFFFFFFu, tau, o));
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    tau = __shfl_sync(0xFFFFFFFFu, tau, 0);
    sum = __shfl_sync(0xFFFFFFFFu, sum, 0);
    const bool fits = __all_sync(0xFFFFFFFFu, listed <= CAND);
    const bool complete = tau == ~0ull;  // the list holds every word that weighs anything
    const int q = warp % CS;             // SW / CS warps fetch each list
    const int nq = min(__shfl_sync(0xFFFFFFFFu, listed, q), CAND);
    __syncthreads();
    const uint32_t from = at_rank(s.cand, q);
    for (int i0 = (warp / CS) * 32; i0 < nq; i0 += SW / CS * 32) {
      const unsigned long long cv = i0 + lane < nq ? peer64(from + 8 * (i0 + lane)) : ~0ull;
      const bool on = cv <= tau && i0 + lane < nq;
      const int at = push_at(&s.nlist, on);
      if (on && at < LIST) s.list[at] = cv;
    }
    __syncthreads();
    const int n = s.nlist;
    bool good = fits && n <= LIST && n > 0 && (k == 0 || by_top_k);
    if (mx == -INFINITY) {  // no word is left
      if (tid == 0) {
        a.ids[m] = -1;
        if (a.probs) a.probs[m] = 0.0f;
        s.done = 1;
      }
    } else if (good) {
      unsigned long long total = sum;  // weight of the words kept
      // first the likeliest words by one warp, then all of the list by the block
      if (n > FEW) sort_list(s, r, n);
      bool found = false;
      if (warp == 0) {
        unsigned long long cv = 0, kept = total;
        found = choose_in_warp(s.list, n > FEW, r, min(n, FEW), complete && n <= FEW, k, p, mp, u, kept, cv);
        if (found && lane == 0) {
          write_row(a, m, r, cv, kept);
          s.done = 1;
        }
      }
      if (n > FEW && !__syncthreads_or(found)) {
        const Held h = hold(s, r, n);
        if (k > 0) {
          if (pass_at(s, h, 0, static_cast<unsigned long long>(k) - 1, true)) {
            total = s.found_before + r.units(logit_of(s.found_cv));
          } else {  // fewer weigh anything: all of them, if they are listed
            good = complete || k <= n;
            unsigned long long t = 0;
#pragma unroll
            for (int i = 0; i < LIST / STH; ++i) t += h.w[i];
            total = block_sum(s, t);
          }
        }
        bool bounded = k > 0;  // the kept words end inside the list
        if (good && p < 1.0f && pass_at(s, h, 0, nucleus(p, total), false)) {
          total = min(total, s.found_before + r.units(logit_of(s.found_cv)));
          bounded = true;
        }
        if (good && mp > 0.0f) {
          unsigned long long t = 0;
          int below = 0;  // some listed word is below min_p
#pragma unroll
          for (int i = 0; i < LIST / STH; ++i) {
            const int j = tid * (LIST / STH) + i;
            if (j < n && r.weight(logit_of(s.list[j])) >= fminf(mp, 1.0f)) t += h.w[i];
            else below |= j < n;
          }
          below = __syncthreads_or(below);
          t = block_sum(s, t);
          if (below || complete) {
            total = min(total, t);
            bounded = true;
          }
        }
        // a nucleus that ends past the list is only harmless if another cut ends inside
        good = good && (bounded || !(p < 1.0f || mp > 0.0f));
        if (good) good = pass_at(s, h, 0, share(u, total), false);
        if (good && tid == 0) {
          write_row(a, m, r, s.found_cv, total);
          s.done = 1;
        }
      }
    }
  }
  cluster_sync();
  const bool done = peer32(at_rank(&s.done, 0)) != 0;
  cluster_sync();
  if (done) return;

  if (tail.rows) {  // left to the clusters of eight that follow
    if (rank == 0 && tid == 0) tail.rows[atomicAdd(tail.count, 1)] = Left{m, r.lmax, sum};
    return;
  }
  whole_row(s, a, row, m, rank, CS, r, by_top_k ? 0 : cluster_mass(s, CS));
}

// The rows that sample_kernel left, by clusters of eight CTAs in turn; the last CTA to leave clears the count.
template <class X>
__global__ void __launch_bounds__(STH, 2) tail_kernel(const __grid_constant__ SampleArgs a, Tail tail) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  const int rank = blockIdx.x % 8, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int n = __ldcg(tail.count);
  for (int i = blockIdx.x / 8; i < n; i += gridDim.x / 8) {
    const Left todo = tail.rows[i];
    const int m = todo.m;
    const X* row = static_cast<const X*>(a.logits) + m * a.row_stride;
    float temp, p, mp, u;
    int k;
    settings(a, m, temp, k, p, mp, u);
    whole_row(s, a, row, m, rank, 8, row_of(todo.lmax, temp), todo.total);
    cluster_sync();
  }
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(tail.left, 1) == static_cast<int>(gridDim.x) - 1) {
      *tail.count = 0;
      *tail.left = 0;
    }
  }
}

}  // namespace

// The workspace: the tail's counters (zero between calls) and its rows.
size_t sample_workspace_bytes(int64_t M, int64_t) { return (256 + static_cast<size_t>(M) * sizeof(Left) + 255) / 256 * 256; }

namespace {
template <class X>
cudaError_t launch_x(const SampleArgs& a, cudaStream_t st) {
  static bool smem_set[64] = {false};
  bool& set = smem_set[current_device_id()];
  if (!set) {
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<X>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(tail_kernel<X>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
    if (e != cudaSuccess) return e;
    set = true;
  }
  // CTAs per row: as many as the device holds at once, two per SM, with at least 4096 words
  // each.
  const int sms = num_sms();
  int CS = 1;
  while (CS < 8 && static_cast<int64_t>(a.M) * CS * 2 <= 2 * sms && a.V / (CS * 2) >= 4096) CS *= 2;
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
  // A row that needs the whole-row path keeps its few CTAs busy long after the others are done: where a row has fewer
  // than eight of them and enough words, those rows are left to a second launch.
  Tail tail = {nullptr, nullptr, nullptr};
  const bool second = CS < 8 && a.V >= 32768;
  if (second) {
    tail.count = static_cast<int*>(a.ws);
    tail.left = tail.count + 1;
    tail.rows = reinterpret_cast<Left*>(tail.count + 64);
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, sample_kernel<X>, a, CS, tail);
  if (e == cudaSuccess && second) {
    cfg.gridDim = dim3(2 * sms / 8 * 8);
    attr[1].val.clusterDim.x = 8;
    e = cudaLaunchKernelEx(&cfg, tail_kernel<X>, a, tail);
  }
  return e;
}
}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int bf16, cudaStream_t st) {
  return bf16 ? launch_x<__nv_bfloat16>(a, st) : launch_x<float>(a, st);
}

}  // namespace kq
