// kq_sample.cu -- the next token of each row of logits, from a given uniform
// number u:  w_i = exp((l_i - l_max) / temperature); the words in descending
// order of their logits (equal ones by index), cut to top_k, then to the
// shortest prefix that holds top_p of the remaining weight, then to the words
// with w_i >= min_p; the token is the first word whose running sum of the kept
// weights exceeds u times their total.
//
// Weights are summed as integers, w_i in units of 2^-40 of the largest: the
// sums are exact, so no order of summation changes a cut or the token (what a
// word below 2^-40 of the likeliest loses is far below the fp32 rounding of
// the likeliest itself), and 2^18 words stay far below 2^64.
//
// One CTA per row.  A cut is found as a key (the logits' bits in an order that
// compares as integers) by bisection over the key's 32 bits, a pass over the
// row each, and the number of words equal to that key that are kept.
#include "kq_cache.h"

namespace kq {
namespace {

constexpr int STH = 1024;

__device__ __forceinline__ float logit(const float* p, int i) { return __ldg(p + i); }
__device__ __forceinline__ float logit(const __nv_bfloat16* p, int i) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p) + i)) << 16);
}
// Order-preserving key: larger logits have larger keys; a NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

struct Sums { unsigned long long mass; int count; };

struct RowCtx {
  float lmax, temp;
  __device__ float weight(uint32_t key) const {
    const float l = value_of(key);
    return l == lmax ? 1.0f : temp > 0.0f ? expf((l - lmax) / temp) : 0.0f;
  }
  __device__ unsigned long long units(uint32_t key) const {
    return static_cast<unsigned long long>(weight(key) * 1099511627776.0f);
  }
};

__device__ Sums block_sum(Sums s) {
  __shared__ unsigned long long sm[STH / 32];
  __shared__ int sc[STH / 32];
  __shared__ Sums tot;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.mass += __shfl_xor_sync(0xFFFFFFFFu, s.mass, o);
    s.count += __shfl_xor_sync(0xFFFFFFFFu, s.count, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) { sm[threadIdx.x >> 5] = s.mass; sc[threadIdx.x >> 5] = s.count; }
  __syncthreads();
  if (threadIdx.x == 0) {
    Sums t = {0, 0};
    for (int i = 0; i < STH / 32; ++i) { t.mass += sm[i]; t.count += sc[i]; }
    tot = t;
  }
  __syncthreads();
  return tot;
}

template <class X>
__device__ Sums sum_at_least(const X* row, int V, const RowCtx& c, uint32_t key) {
  Sums s = {0, 0};
  for (int i = threadIdx.x; i < V; i += STH) {
    const uint32_t k = key_of(logit(row, i));
    if (k >= key) { s.mass += c.units(k); s.count += 1; }
  }
  return block_sum(s);
}

// The largest key whose words and those above them hold more than x (of mass, or of count).
template <class X>
__device__ uint32_t crossing(const X* row, int V, const RowCtx& c, unsigned long long x, bool mass) {
  uint32_t key = 0;
  for (int b = 31; b >= 0; --b) {
    const uint32_t t = key | (1u << b);
    const Sums s = sum_at_least(row, V, c, t);
    if ((mass ? s.mass : static_cast<unsigned long long>(s.count)) > x) key = t;
  }
  return key;
}

template <class X>
__global__ void __launch_bounds__(STH) sample_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ float s_max[STH / 32];
  __shared__ int s_scan[STH];
  pdl_wait();
  pdl_launch_dependents();
  const int m = blockIdx.x, V = a.V;
  const X* row = static_cast<const X*>(a.logits) + m * a.row_stride;
  RowCtx c;
  c.temp = a.temperature ? a.temperature[m] : 1.0f;
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < V; i += STH) mx = fmaxf(mx, logit(row, i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
  for (int i = 0; i < STH / 32; ++i) mx = fmaxf(mx, s_max[i]);
  c.lmax = mx;
  if (mx == -INFINITY) {  // no word is left
    if (threadIdx.x == 0) {
      a.ids[m] = -1;
      if (a.probs) a.probs[m] = 0.0f;
    }
    return;
  }
  const bool greedy = !(c.temp > 0.0f);
  // top_k: the kept words are those above `key`, and the first `ties` equal to it
  int k = greedy ? 1 : a.top_k ? a.top_k[m] : 0;
  if (k <= 0 || k > V) k = V;
  unsigned long long total;  // of the kept words
  {
    const uint32_t key = crossing(row, V, c, static_cast<unsigned long long>(k) - 1, false);
    Sums above = {0, 0};
    if (key != 0xFFFFFFFFu) above = sum_at_least(row, V, c, key + 1);
    total = above.mass + (k - above.count) * c.units(key);
  }
  const float p = a.top_p ? a.top_p[m] : 1.0f;
  if (p < 1.0f) {
    const double want = static_cast<double>(p) * static_cast<double>(total);
    // kept: the words with less than `want` before them
    unsigned long long x = want > 1.0 ? static_cast<unsigned long long>(ceil(want)) - 1 : 0;
    if (x >= total) x = total - 1;
    const uint32_t key = crossing(row, V, c, x, true);
    Sums above = {0, 0};
    if (key != 0xFFFFFFFFu) above = sum_at_least(row, V, c, key + 1);
    const unsigned long long w = c.units(key), t = above.mass + ((x - above.mass) / w + 1) * w;
    total = t < total ? t : total;
  }
  const float mp = a.min_p ? a.min_p[m] : 0.0f;
  if (mp > 0.0f) {
    Sums s = {0, 0};
    for (int i = threadIdx.x; i < V; i += STH) {
      const uint32_t kk = key_of(logit(row, i));
      const float w = c.weight(kk);
      if (w >= mp || w == 1.0f) s.mass += c.units(kk);
    }
    s = block_sum(s);
    total = s.mass < total ? s.mass : total;
  }
  const double uw = static_cast<double>(a.u[m]) * static_cast<double>(total);
  unsigned long long x = uw > 0.0 ? static_cast<unsigned long long>(uw) : 0;
  if (x >= total) x = total - 1;
  const uint32_t key = crossing(row, V, c, x, true);
  Sums above = {0, 0};
  if (key != 0xFFFFFFFFu) above = sum_at_least(row, V, c, key + 1);
  int nth = static_cast<int>((x - above.mass) / c.units(key));  // among the words equal to key, by index
  // each thread's words are consecutive here
  const int per = (V + STH - 1) / STH, i0 = threadIdx.x * per, i1 = min(V, i0 + per);
  int n = 0;
  for (int i = i0; i < i1; ++i) n += key_of(logit(row, i)) == key;
  s_scan[threadIdx.x] = n;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < static_cast<int>(threadIdx.x); ++i) before += s_scan[i];
  if (nth >= before && nth < before + n) {
    for (int i = i0; i < i1; ++i)
      if (key_of(logit(row, i)) == key && before++ == nth) {
        a.ids[m] = i;
        if (a.probs) a.probs[m] = static_cast<float>(static_cast<double>(c.units(key)) / static_cast<double>(total));
      }
  }
}

}  // namespace

size_t sample_workspace_bytes(int64_t, int64_t) { return 256; }

cudaError_t launch_sample(const SampleArgs& a, int bf16, cudaStream_t st) {
  if (bf16) return launch_pdl(sample_kernel<__nv_bfloat16>, dim3(a.M), dim3(STH), 0, st, a);
  return launch_pdl(sample_kernel<float>, dim3(a.M), dim3(STH), 0, st, a);
}

}  // namespace kq
