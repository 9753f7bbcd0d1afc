// kq_vec.cuh -- loads and stores of the cache writers (kq_append.cu,
// kq_latent_append.cu): four values at a time as fp32, rounded once to the
// stored type (e4m3: saturated, a NaN stays a NaN).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

namespace kq {

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 bf16x4(uint2 u) {
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) { return bf16x4(__ldg(reinterpret_cast<const uint2*>(p))); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
}
__device__ __forceinline__ uint32_t e4m3x4(float4 v) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z, v.w), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void store4(__nv_fp8_e4m3* p, float4 v) { *reinterpret_cast<uint32_t*>(p) = e4m3x4(v); }
// Eight neighbouring values.
struct F8 {
  float4 a, b;
};
__device__ __forceinline__ F8 load8(const float* p) { return {load4(p), load4(p + 4)}; }
__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  return {bf16x4(make_uint2(u.x, u.y)), bf16x4(make_uint2(u.z, u.w))};
}
__device__ __forceinline__ void store8(float* p, F8 v) {
  store4(p, v.a);
  store4(p + 4, v.b);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, F8 v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v.a.x, v.a.y), bf16_pair(v.a.z, v.a.w), bf16_pair(v.b.x, v.b.y),
                                            bf16_pair(v.b.z, v.b.w));
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, F8 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(v.a), e4m3x4(v.b));
}
__device__ __forceinline__ float sq4(float4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }
__device__ __forceinline__ float4 scale4(float4 v, float s, float4 w, float off) {
  return make_float4(v.x * s * (w.x + off), v.y * s * (w.y + off), v.z * s * (w.z + off), v.w * s * (w.w + off));
}
__device__ __forceinline__ float4 over4(float4 v, float s) { return make_float4(v.x / s, v.y / s, v.z / s, v.w / s); }

// (a, b) -> (a c - b s, b c + a s) of the four pairs that x0 and x1 hold: x0[i] with x1[i], or (interleaved) neighbours.
__device__ __forceinline__ void rotate8(float4& x0, float4& x1, float4 c, float4 s, bool interleaved) {
  const float4 p = x0, q = x1;
  if (interleaved) {  // pairs (p.x, p.y), (p.z, p.w), (q.x, q.y), (q.z, q.w)
    x0 = make_float4(p.x * c.x - p.y * s.x, p.y * c.x + p.x * s.x, p.z * c.y - p.w * s.y, p.w * c.y + p.z * s.y);
    x1 = make_float4(q.x * c.z - q.y * s.z, q.y * c.z + q.x * s.z, q.z * c.w - q.w * s.w, q.w * c.w + q.z * s.w);
  } else {
    x0 = make_float4(p.x * c.x - q.x * s.x, p.y * c.y - q.y * s.y, p.z * c.z - q.z * s.z, p.w * c.w - q.w * s.w);
    x1 = make_float4(q.x * c.x + p.x * s.x, q.y * c.y + p.y * s.y, q.z * c.z + p.z * s.z, q.w * c.w + p.w * s.w);
  }
}

}  // namespace kq
