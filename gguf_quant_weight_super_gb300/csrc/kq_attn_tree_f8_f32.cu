// kq_attn_tree_f8_f32.cu -- the attention kernel's instantiations for trees of drafted tokens, e4m3 caches and fp32 queries.
#include "kq_attn_kernel.cuh"

namespace kq {

cudaError_t launch_attn_tree_f8_f32(const attn::Params& p, int rows, cudaStream_t st) {
  return attn::launch_kind<float, __nv_fp8_e4m3, true>(p, rows, st, nullptr);
}

}  // namespace kq
