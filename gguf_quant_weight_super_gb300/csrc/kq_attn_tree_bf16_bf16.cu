// kq_attn_tree_bf16_bf16.cu -- the attention kernel's instantiations for trees of drafted tokens, bf16 caches and bf16 queries.
#include "kq_attn_kernel.cuh"

namespace kq {

cudaError_t launch_attn_tree_bf16_bf16(const attn::Params& p, int rows, cudaStream_t st) {
  return attn::launch_kind<__nv_bfloat16, __nv_bfloat16, true>(p, rows, st, nullptr);
}

}  // namespace kq
