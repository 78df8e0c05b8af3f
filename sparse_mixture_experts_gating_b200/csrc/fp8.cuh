// Device helpers of the 8-bit operators.
#pragma once

#include <stdint.h>

namespace moe {

// The scale of a block with largest magnitude m, and the factor that takes its
// values to codes (both one IEEE division).
struct Fp8Scale {
  float scale, inv;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float m) {
  const float a = fmaxf(m, 7.8886090522101181e-31f);  // 2^-100
  Fp8Scale q;
  q.scale = __fdiv_rn(a, 448.f);
  q.inv = __fdiv_rn(448.f, a);
  return q;
}

// Two fp32 values as e4m3 codes, `a` in the low byte (nearest, ties to even; beyond +-448 saturates).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

}  // namespace moe
