// Packed pairs of fp32: one instruction for two elements.  The training
// operators' kernels are bound by instruction issue as soon as they are not
// by HBM.
#pragma once
#include "ptx.cuh"

namespace ibwd {

__device__ __forceinline__ uint64_t bits2(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  const uint64_t d = mul_f32x2(bits2(a), bits2(b));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  const uint64_t d = fma_f32x2(bits2(a), bits2(b), bits2(c));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

}  // namespace ibwd
