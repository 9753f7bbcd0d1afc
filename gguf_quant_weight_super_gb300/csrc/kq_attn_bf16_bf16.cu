// kq_attn_bf16_bf16.cu -- the attention kernel's instantiations for bf16 caches and bf16 queries.
#include "kq_attn_kernel.cuh"

namespace kq {

cudaError_t launch_attn_bf16_bf16(const attn::Params& p, int rows, cudaStream_t st, AttnShape* ask) {
  return attn::launch_kind<__nv_bfloat16, __nv_bfloat16>(p, rows, st, ask);
}

}  // namespace kq
