// kq_cache.h -- declarations shared by the operators around the paged
// key-value cache (kq_append.cu, kq_attn.cu) and by the sampler (kq_sample.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/kq.h"
#include "kq_internal.h"

namespace kq {

// Device error codes of these operators (beside kq_ptx.cuh's).
enum : int {
  DEV_ERR_PAGE = 4,      // a page id outside [0, n_pages), or a length past the page table
  DEV_ERR_POSITION = 5,  // a position outside the rotary table
};

constexpr int kMaxHeadDim = 256;
inline bool head_dim_supported(int d) { return d == 64 || d == 128 || d == 256; }

// ---- trees of drafted tokens: the T <= 64 newest slots of a sequence hold a tree, a 64-bit mask per token says which of
// them it sees.  Slots before the sequence's start hold nothing: their bits do not count, their tokens are padding.
constexpr int kMaxTree = 64;
__device__ __forceinline__ uint64_t tree_there(int T, int len) {
  const uint64_t all = ~0ull >> (64 - T);
  return len >= T ? all : len > 0 ? all & ~0ull << (T - len) : 0;
}
// What token t sees of the drafted tokens (0: it is padding).
__device__ __forceinline__ uint64_t tree_bits(uint64_t mask, int T, int t, int len) {
  const uint64_t there = tree_there(T, len);
  return there >> t & 1 ? mask & there : 0;
}
// Its position: the tokens that it sees stand in a row after the context.  -1: padding.
__device__ __forceinline__ int tree_position(uint64_t bits, int T, int len) {
  return bits ? max(len - T, 0) + __popcll(bits) - 1 : -1;
}

struct AppendArgs {
  kq_kv_cache c;
  kq_rope rope;
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* seq_lens;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  void* q_out;
  int B, T, Hq;
  int page_shift;
  int* err;
  const uint64_t* tree;  // [B][T] masks, or NULL: a chain
};
cudaError_t launch_kv_append(const AppendArgs& a, int x_bf16, int out_bf16, cudaStream_t st);

struct AttnArgs {
  kq_kv_cache c;
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* seq_lens;
  const void* q;
  int64_t q_stride;
  void* out;
  float scale, softcap;
  int window;
  int B, T, Hq, G;
  int page_shift;
  int room;  // positions that a sequence can have
  void* ws;
  int* err;
  const uint64_t* tree;  // [B][T] masks, or NULL: a chain
};
constexpr int kMaxSeqs = 4096;  // sequences of an attention call, whose place in the line of tiles lies in shared memory
// Positions are counted in 32 bits, tiles and copies ahead of the last one included.
constexpr int64_t kMaxPositions = INT32_MAX - 4095;
size_t attn_workspace_bytes(int head_dim, int Hkv, int64_t T, int Hq);
size_t attn_tree_workspace_bytes(int head_dim, int Hkv, int64_t T, int Hq);
// With `ask`: no launch, but the CTAs per SM that the kernel is laid out for and that the device holds at once.
struct AttnShape {
  int planned, resident;
};
cudaError_t launch_attn(const AttnArgs& a, int q_bf16, cudaStream_t st, AttnShape* ask = nullptr);

// A verified tree's walk, and the accepted branch's slots of up to kMaxPools pools of one geometry (strides in bytes).
constexpr int kMaxPools = 256;
struct TreeArgs {
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* seq_lens;
  const uint64_t* tree;
  const int32_t *tokens, *ids;
  int32_t *path, *count, *next, *new_lens;
  int B, T;
  int page_shift;
  int* err;
  int64_t n_pages, page_stride, slot_stride, head_stride;
  int n_pools, cols, head_cols;  // 16-byte columns of a slot, and of one of its heads
  void* pool[kMaxPools];
};
cudaError_t launch_tree_accept(const TreeArgs& a, cudaStream_t st);

struct LatentAppendArgs {
  kq_latent_cache l;
  kq_rope rope;
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* seq_lens;
  const uint64_t* tree;  // or NULL
  const void *q_latent, *q_rope, *c;
  int64_t q_latent_stride, q_rope_stride, q_rope_head_stride, c_stride;
  void* q_out;
  int B, T, H;
  int page_shift;
  int* err;
};
cudaError_t launch_latent_append(const LatentAppendArgs& a, int x_bf16, cudaStream_t st);

struct LatentArgs {
  kq_latent_cache l;
  const int32_t* page_table;
  int64_t max_pages;
  const int32_t* seq_lens;
  const uint64_t* tree;  // or NULL
  const void* q;
  int64_t q_stride;
  void* out;
  float scale;
  int B, T, H;
  int page_shift;
  int room;  // positions that a sequence can have
  void* ws;
  int* err;
};
size_t latent_workspace_bytes(const kq_latent_cache& l, int64_t T, int H);
cudaError_t launch_latent(const LatentArgs& a, cudaStream_t st);

struct SampleArgs {
  const void* logits;
  int64_t row_stride;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t* ids;
  float* probs;
  void* ws;
  int M, V;
};
size_t sample_workspace_bytes(int64_t M, int64_t V);
cudaError_t launch_sample(const SampleArgs& a, int bf16, cudaStream_t st);

// Launch with programmatic stream serialization, as every product is.
template <class... P, class... A>
inline cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kq
