// kq_tree.cu -- what follows a verified tree of drafted tokens, in one launch
// for all layers: the walk along the branch that the model's words accept, and
// the move of that branch's cache slots to where a chain's would lie.
//
// The walk needs ids -> child -> ids -> ..., at most T steps of a ballot over
// the tokens, whose masks, words and model's words one warp holds in
// registers.  Every CTA walks for itself (the T tokens' data come from L2 in one
// round trip), which costs less than a second launch or a grid barrier.
//
// The move.  The branch 0 = p_0 < p_1 < ... goes from slots base + p_i to base + i.
// As p_i >= i and the branch ascends, slot i is no later source p_k > p_i >= i:
// a thread that moves its 16 bytes of a slot for all i in order, loads of a batch
// before its stores, needs no other thread's order.  Two rows of bytes per
// accepted token and layer are nothing beside the latency of length -> masks ->
// walk -> page -> load -> store, so the columns of 16 bytes are spread over as
// many threads as there are.  Measured on one GB300, calls in a graph: 16 nodes,
// 36 layers of 8 heads of 128, bf16, 3.1 us; 32 x 61 nodes, 30 layers of 4 heads
// of 256, e4m3, 4.4 us.
#include "kq_cache.h"

namespace kq {
namespace {

constexpr int MTH = 256;  // threads per CTA, a column of 16 bytes each
constexpr int BATCH = 8;  // loads in flight per thread

struct Walk {
  int path[kMaxTree];
  int n, next, base;
};

// One warp: lane l holds tokens l and l + 32.
__device__ __forceinline__ void walk(const TreeArgs& a, int b, int len, Walk& w) {
  const int lane = threadIdx.x;
  uint64_t bits[2];
  int word[2], id[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    const int64_t at = static_cast<int64_t>(b) * a.T + t;
    bits[i] = t < a.T ? __ldg(a.tree + at) : 0;
    word[i] = t < a.T ? __ldg(a.tokens + at) : 0;
    id[i] = t < a.T ? __ldg(a.ids + at) : 0;
    if (t < a.T) bits[i] = tree_bits(bits[i], a.T, t, len);
  }
  auto bits_at = [&](int t) { return __shfl_sync(0xFFFFFFFFu, t < 32 ? bits[0] : bits[1], t & 31); };
  auto id_at = [&](int t) { return __shfl_sync(0xFFFFFFFFu, t < 32 ? id[0] : id[1], t & 31); };
  int n = 0, cur = 0, next = -1;
  uint64_t seen = bits_at(0);
  if (seen & 1) {
    for (;;) {
      if (lane == 0) w.path[n] = cur;
      ++n;
      next = id_at(cur);
      // children come after their parent and see what it sees and themselves
      uint32_t hit[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        hit[i] = __ballot_sync(0xFFFFFFFFu, t > cur && bits[i] == (seen | 1ull << t) && word[i] == next);
      }
      if ((hit[0] | hit[1]) == 0) break;
      cur = hit[0] ? __ffs(hit[0]) - 1 : 32 + __ffs(hit[1]) - 1;
      seen = bits_at(cur);
    }
  }
  if (lane == 0) {
    w.n = n;
    w.next = next;
    w.base = max(len - a.T, 0);
  }
}

__global__ void __launch_bounds__(MTH) tree_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ Walk w;
  __shared__ int64_t from[kMaxTree], to[kMaxTree];  // bytes from a pool's start; from -1: stays
  __shared__ int moves;
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int len = max(__ldg(a.seq_lens + b), 0);
  if (tid < 32) walk(a, b, len, w);
  __syncthreads();
  if (blockIdx.x == 0) {
    if (a.path)
      for (int t = tid; t < a.T; t += MTH) a.path[static_cast<int64_t>(b) * a.T + t] = t < w.n ? w.path[t] : -1;
    if (tid == 0) {
      if (a.count) a.count[b] = w.n;
      if (a.next) a.next[b] = w.next;
      if (a.new_lens) a.new_lens[b] = w.base + w.n;
    }
  }
  if (a.n_pools == 0) return;
  if (tid < 32) {  // the slots that move, in order
    int m = 0;
    for (int i0 = 0; i0 < w.n; i0 += 32) {
      const int i = i0 + tid;
      bool go = i < w.n && w.path[min(i, kMaxTree - 1)] != i;
      int64_t off[2] = {0, 0};
      if (go) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t j = static_cast<int64_t>(w.base) + (e ? i : w.path[i]);
          const int64_t pi = j >> a.page_shift;
          const int page = pi < a.max_pages ? __ldg(a.page_table + b * a.max_pages + pi) : -1;
          if (page < 0 || page >= a.n_pages) {
            record_error(a.err, DEV_ERR_PAGE);
            go = false;
          } else {
            off[e] = page * a.page_stride + (j & ((1 << a.page_shift) - 1)) * a.slot_stride;
          }
        }
      }
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, go);
      if (go) {
        const int at = m + __popc(who & ((1u << tid) - 1));
        from[at] = off[0];
        to[at] = off[1];
      }
      m += __popc(who);
    }
    if (tid == 0) moves = m;
  }
  __syncthreads();
  const int col = blockIdx.x * MTH + tid;
  if (moves == 0 || col >= a.n_pools * a.cols) return;
  const int pool = col / a.cols, c = col - pool * a.cols, head = c / a.head_cols;
  uint8_t* mem = static_cast<uint8_t*>(a.pool[pool]) + head * a.head_stride + (c - head * a.head_cols) * 16;
  for (int i0 = 0; i0 < moves; i0 += BATCH) {
    uint4 v[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < moves) v[i] = *reinterpret_cast<const uint4*>(mem + from[i0 + i]);
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < moves) *reinterpret_cast<uint4*>(mem + to[i0 + i]) = v[i];
  }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeArgs& a, cudaStream_t st) {
  const int64_t cols = static_cast<int64_t>(a.n_pools) * a.cols;
  const int64_t grid = cols > 0 ? (cols + MTH - 1) / MTH : 1;
  return launch_pdl(tree_kernel, dim3(static_cast<unsigned>(grid), a.B), dim3(MTH), 0, st, a);
}

}  // namespace kq
