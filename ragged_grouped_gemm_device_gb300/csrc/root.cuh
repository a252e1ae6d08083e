// The square root of AdamW's second moments.
#pragma once

namespace moe {
namespace {

// The square root of a value in [2^-126, inf): an estimate s from the reciprocal root y, and Newton's step s + (v - s^2) y / 2 with
// the residual from a fused product. It equals sqrtf as long as the residual is a normal number, v from 2^-80 on; below that it is
// within a unit (a test compares all values). Of zeros, subnormals, infinities and NaNs it is not finite. It takes a quarter of sqrtf's
// instructions.
__device__ __forceinline__ float sqrt_normal(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  const float s = __fmul_rn(v, y);
  return __fmaf_rn(__fmaf_rn(-s, s, v), 0.5f * y, s);
}

}  // namespace
}  // namespace moe
