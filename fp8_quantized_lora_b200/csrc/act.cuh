// The activations of the linear layer's epilogue and their derivatives, in
// float32.
//   ReLU       max(z, 0)                        derivative 1 where z > 0, else 0
//   GELU       z Phi(z), Phi the normal CDF     Phi(z) + z phi(z)
//   GELU tanh  z p, p = 1 / (1 + exp(-2u)),     p + z p (1 - p) 2u',
//              u = sqrt(2/pi)(z + 0.044715 z^3) u' = sqrt(2/pi)(1 + 0.134145 z^2)
//   SiLU       z p, p = 1 / (1 + exp(-z))       p + z p (1 - p)
// ((1 + tanh u) / 2 is the logistic function of 2u, so both sigmoid forms
// share one exponential and one division.)
#pragma once

#include <cstdint>

#include "../../include/falqon.h"

namespace falqon {

// 1 / (1 + exp(-t)).  exp overflows to infinity for t < -88: the quotient is
// then 0, the limit.
__device__ __forceinline__ float logistic(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

constexpr float kGeluTwoU = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (kAct == FALQON_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
  if constexpr (kAct == FALQON_ACT_GELU_ERF) return 0.5f * z * erfcf(-kInvSqrt2 * z);
  if constexpr (kAct == FALQON_ACT_GELU_TANH) return z * logistic(kGeluTwoU * (z + kGeluCubic * z * z * z));
  if constexpr (kAct == FALQON_ACT_SILU) return z * logistic(z);
  return z;
}

// p + z u p (1 - p) for p = 1 / (1 + exp(-t)): with e = exp(-|t|) <= 1 and
// r = 1 / (1 + e), p is r or e r and p (1 - p) = e r^2, so neither tail
// cancels or overflows.
__device__ __forceinline__ float logistic_slope(float t, float zu) {
  const float e = __expf(-fabsf(t));
  const float r = __fdividef(1.0f, 1.0f + e);
  const float q = e * r;
  return fmaf(zu * q, r, t < 0.0f ? q : r);
}

template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (kAct == FALQON_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (kAct == FALQON_ACT_GELU_ERF)
    return 0.5f * erfcf(-kInvSqrt2 * z) + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
  if constexpr (kAct == FALQON_ACT_GELU_TANH) {
    const float z2 = fminf(z * z, 400.0f);  // past |z| = 20 p is 0 or 1 whatever z: keeps the products finite
    return logistic_slope(kGeluTwoU * z * (1.0f + kGeluCubic * z2), z * (kGeluTwoU * (1.0f + 3.0f * kGeluCubic * z2)));
  }
  if constexpr (kAct == FALQON_ACT_SILU) return logistic_slope(z, z);
  return 1.0f;
}

}  // namespace falqon
