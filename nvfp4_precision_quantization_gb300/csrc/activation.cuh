// activation.cuh -- the layer operators' activations and their derivatives (FP32).
//
// GELU's tanh form is z p with p = 1 / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
// (1 + tanh u = 2 p), SILU is z p with p = 1 / (1 + exp(-z)): one exponential and one
// reciprocal each, whose relative errors (a few 2^-23, times |z| for the exponent's
// product) fall on p where it is not already saturated.
#pragma once

#include "device_common.cuh"

namespace nvfp4 {

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// m with the sign of z (m >= 0)
__device__ __forceinline__ float with_sign(float m, float z) {
  return __uint_as_float(__float_as_uint(m) | (__float_as_uint(z) & 0x80000000u));
}

// act'(z) of a pair, and its value.  GELU and SILU are z p(u), p = 1 / (1 + exp(-u)), u odd in z,
// so with a = |z|, t = exp(-u(a)) <= 1 and r = 1 / (1 + t) = p(u(a)):
//   act' = 1/2 + sgn(z) (r - 1/2 + a t r^2 u'(a)),   act = z r (z >= 0) or z t r,
// where p (1 - p) = t r^2 is never the difference of 1 and a rounded p (it is multiplied by
// a u' of up to 100 before it vanishes).  a is cut at 64, where t is 0 or below 2^-92, so that
// 0 never meets an infinite u' (and the value of a z below -64 is 0); a NaN stays one.
template <int ACT>
__device__ __forceinline__ Pair act_slope(Pair z, Pair& value) {
  if constexpr (ACT == kActRelu) {
    value = {z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y};  // NaN stays
    return {z.x > 0.0f ? 1.0f : 0.0f, z.y > 0.0f ? 1.0f : 0.0f};
  }
  if constexpr (ACT != kActGelu && ACT != kActSilu) {
    value = z;
    return {1.0f, 1.0f};
  }
  constexpr float kLog2e = 1.4426950408889634f;
  Pair a;
  asm("min.NaN.f32 %0, %1, 0f42800000;" : "=f"(a.x) : "f"(fabsf(z.x)));
  asm("min.NaN.f32 %0, %1, 0f42800000;" : "=f"(a.y) : "f"(fabsf(z.y)));
  Pair w, du;  // u(a) log2(e), u'(a)
  if constexpr (ACT == kActGelu) {
    constexpr float c0 = kGelu2C * kLog2e, c1 = kGelu2C * kGeluA * kLog2e;
    constexpr float d1 = 3.0f * kGelu2C * kGeluA;
    const Pair a2 = pair_mul(a, a);
    w = pair_mul(a, pair_fma({c1, c1}, a2, {c0, c0}));
    du = pair_fma({d1, d1}, a2, {kGelu2C, kGelu2C});
  } else {
    w = pair_mul(a, {kLog2e, kLog2e});
    du = {1.0f, 1.0f};
  }
  const Pair t = {ex2_approx(-w.x), ex2_approx(-w.y)};
  const Pair one_t = pair_add(t, {1.0f, 1.0f});
  const Pair r = {rcp_approx(one_t.x), rcp_approx(one_t.y)};
  const Pair tr = pair_mul(t, r);
  value = pair_mul(z, {z.x < 0.0f ? (z.x < -64.0f ? 0.0f : tr.x) : r.x,
                       z.y < 0.0f ? (z.y < -64.0f ? 0.0f : tr.y) : r.y});
  const Pair q = pair_mul(tr, r);
  Pair aq = pair_mul(a, q);
  if constexpr (ACT == kActGelu) aq = pair_mul(aq, du);
  const Pair m = pair_add(pair_add(r, {-0.5f, -0.5f}), aq);
  return pair_add({with_sign(m.x, z.x), with_sign(m.y, z.y)}, {0.5f, 0.5f});
}
template <int ACT>
__device__ __forceinline__ Pair act_slope(Pair z) {
  Pair value;
  return act_slope<ACT>(z, value);
}

// act(z) of a pair: z p with p = 1 / (1 + 2^-w), w = u log2(e).
template <int ACT>
__device__ __forceinline__ Pair act_value(Pair z) {
  if constexpr (ACT == kActGelu || ACT == kActSilu) {
    constexpr float kLog2e = 1.4426950408889634f;
    Pair w;
    if constexpr (ACT == kActGelu) {
      constexpr float c0 = kGelu2C * kLog2e, c1 = kGelu2C * kGeluA * kLog2e;
      w = pair_mul(z, pair_fma({c1, c1}, pair_mul(z, z), {c0, c0}));
    } else {
      w = pair_mul(z, {kLog2e, kLog2e});
    }
    const Pair t = pair_add({ex2_approx(-w.x), ex2_approx(-w.y)}, {1.0f, 1.0f});
    return pair_mul(z, {rcp_approx(t.x), rcp_approx(t.y)});
  } else if constexpr (ACT == kActRelu) {
    return {z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y};  // NaN stays
  } else {
    return z;
  }
}

// v[0 .. N) = act(v), the activation known at run time.
template <int ACT, int N>
__device__ __forceinline__ void apply_act_as(float* v) {
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const Pair r = act_value<ACT>(Pair{v[j], v[j + 1]});
    v[j] = r.x;
    v[j + 1] = r.y;
  }
}
template <int N>
__device__ __forceinline__ void apply_act(int act, float* v) {
  if (act == kActRelu) apply_act_as<kActRelu, N>(v);
  else if (act == kActGelu) apply_act_as<kActGelu, N>(v);
  else if (act == kActSilu) apply_act_as<kActSilu, N>(v);
}

}  // namespace nvfp4
