// Two fp32 values computed together, one instruction on sm_100 and up.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace gbo {

__device__ __forceinline__ uint64_t as_bits(float2 a) { return *reinterpret_cast<uint64_t *>(&a); }
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_bits(a)), "l"(as_bits(b)), "l"(as_bits(c)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_bits(a)), "l"(as_bits(b)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_bits(a)), "l"(as_bits(b)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 f2_of(float a) { return make_float2(a, a); }

}  // namespace gbo
