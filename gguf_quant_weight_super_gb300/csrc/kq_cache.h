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
};
// Positions are counted in 32 bits, tiles and copies ahead of the last one included.
constexpr int64_t kMaxPositions = INT32_MAX - 4095;
size_t attn_workspace_bytes(int head_dim, int Hkv, int64_t T, int Hq);
// With `ask`: no launch, but the CTAs per SM that the kernel is laid out for and that the device holds at once.
struct AttnShape {
  int planned, resident;
};
cudaError_t launch_attn(const AttnArgs& a, int q_bf16, cudaStream_t st, AttnShape* ask = nullptr);

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
