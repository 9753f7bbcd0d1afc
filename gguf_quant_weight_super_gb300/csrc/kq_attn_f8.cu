// kq_attn_f8.cu -- the attention kernel's instantiations for e4m3 caches.
#include "kq_attn_kernel.cuh"

namespace kq {

using namespace attn;

namespace {
template <class Q>
cudaError_t launch_q(const Params& p, int rows, cudaStream_t st) {
  switch (p.a.c.head_dim) {
    case 64: return rows == 16 ? launch_one<Q, __nv_fp8_e4m3, 64, 1>(p, st) : launch_one<Q, __nv_fp8_e4m3, 64, 2>(p, st);
    case 128: return rows == 16 ? launch_one<Q, __nv_fp8_e4m3, 128, 1>(p, st) : launch_one<Q, __nv_fp8_e4m3, 128, 2>(p, st);
    default: return launch_one<Q, __nv_fp8_e4m3, 256, 1>(p, st);
  }
}
}  // namespace

cudaError_t launch_attn_f8(const Params& p, int q_bf16, int rows, cudaStream_t st) {
  return q_bf16 ? launch_q<__nv_bfloat16>(p, rows, st) : launch_q<float>(p, rows, st);
}

}  // namespace kq
