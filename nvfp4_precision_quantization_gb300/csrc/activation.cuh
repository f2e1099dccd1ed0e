// activation.cuh -- the layer operators' activations and their derivatives (FP32).
//
// GELU's tanh form is z p with p = 1 / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
// (1 + tanh u = 2 p), SILU is z p with p = 1 / (1 + exp(-z)): one exponential and one
// reciprocal each, whose relative errors (a few 2^-23, times |z| for the exponent's
// product) fall on p where it is not already saturated.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float sigmoid_fast(float x) {
  return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-x)));
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;  // NaN stays
  if constexpr (ACT == kActGelu) {
    const float z2 = __fmul_rn(z, z);
    const float u2 = __fmul_rn(z, __fmaf_rn(kGelu2C * kGeluA, z2, kGelu2C));
    return __fmul_rn(z, sigmoid_fast(u2));
  }
  if constexpr (ACT == kActSilu) return __fmul_rn(z, sigmoid_fast(z));
  return z;
}

// p = 1 / (1 + exp(-x)) and q = p (1 - p) from t = exp(-|x|) <= 1: 1 - p is t / (1 + t) for
// positive x, never the difference of 1 and a rounded p (GELU's slope multiplies q by up
// to z u' of about 100 before q vanishes).
__device__ __forceinline__ void sigmoid_pair(float x, float& p, float& q) {
  const float t = __expf(-fabsf(x));
  const float r = __fdividef(1.0f, __fadd_rn(1.0f, t));
  const float tr = __fmul_rn(t, r);
  p = x >= 0.0f ? r : tr;
  q = __fmul_rn(r, tr);
}

// d act / d z = p + z p (1 - p) u' with u' bounded: where z^2 > 10^4 the factor p (1 - p) is
// 0 and must not meet an infinite u'.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  float p, q;
  if constexpr (ACT == kActGelu) {
    const float z2 = fminf(__fmul_rn(z, z), 1e4f);
    sigmoid_pair(__fmul_rn(z, __fmaf_rn(kGelu2C * kGeluA, z2, kGelu2C)), p, q);
    const float du = __fmaf_rn(3.0f * kGelu2C * kGeluA, z2, kGelu2C);
    return __fmaf_rn(__fmul_rn(z, q), du, p);
  }
  if constexpr (ACT == kActSilu) {
    sigmoid_pair(z, p, q);
    return __fmaf_rn(z, q, p);
  }
  return 1.0f;
}

}  // namespace nvfp4
