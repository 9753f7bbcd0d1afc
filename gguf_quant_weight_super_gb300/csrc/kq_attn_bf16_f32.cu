// kq_attn_bf16_f32.cu -- the attention kernel's instantiations for bf16 caches and fp32 queries.
#include "kq_attn_kernel.cuh"

namespace kq {

cudaError_t launch_attn_bf16_f32(const attn::Params& p, int rows, cudaStream_t st, AttnShape* ask) {
  return attn::launch_kind<float, __nv_bfloat16>(p, rows, st, ask);
}

}  // namespace kq
