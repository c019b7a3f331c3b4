// The activations of the linear layer's epilogue and their derivatives, in
// float32.
//   ReLU       max(z, 0)                        derivative 1 where z > 0, else 0
//   GELU       z Phi(z), Phi the normal CDF     Phi(z) + z phi(z)
//   GELU tanh  z p, p = 1 / (1 + exp(-2u)),     p + z p (1 - p) 2u',
//              u = sqrt(2/pi)(z + 0.044715 z^3) u' = sqrt(2/pi)(1 + 0.134145 z^2)
//   SiLU       z p, p = 1 / (1 + exp(-z))       p + z p (1 - p)
// ((1 + tanh u) / 2 is the logistic function of 2u.)
//
// The kernels that use them are bound by their instructions as much as by
// memory (an epilogue warp spends about 30 a value), so each is written with
// one exp2 and one reciprocal of the special function unit, both off by at
// most 2^-22 relative, subnormal results taken as 0.  Phi comes from the same
// two: Phi(-|z|) = erfc(|z| / sqrt 2) / 2 = exp(-z^2/2) t P(t) / 2 with
// t = 1 / (1 + 0.44 |z| / sqrt 2) and P of degree 7, fitted here by iterated
// least squares to erfc(x) exp(x^2) on 0 <= x <= 14 (relative error below
// 2e-7), so the tail keeps its relative accuracy; erfcf took 45.5 us where
// this took 28.2 us (backward, 4096 x 4096; 20.4 us with two values an
// instruction).
#pragma once

#include <cstdint>

#include "../../include/falqon.h"
#include "elem.cuh"

namespace falqon {

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two values held to [-bound, bound]; NaN for NaN.
__device__ __forceinline__ float2 clamp2(float2 z, float bound) {
  float2 y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(z.x), "f"(bound));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(z.y), "f"(bound));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(y.x), "f"(-bound));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(y.y), "f"(-bound));
  return y;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluTwoU = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// P: the coefficients of t^0 .. t^7.
__host__ __device__ constexpr float tail_coef(int k) {
  return k == 0   ? 0.248216525f
         : k == 1 ? 0.248935506f
         : k == 2 ? 0.21693407f
         : k == 3 ? 0.216996044f
         : k == 4 ? -0.0222996026f
         : k == 5 ? 0.298873633f
         : k == 6 ? -0.279156834f
                  : 0.0715008602f;
}

// t P(t): erfc(|z| / sqrt 2) without its factor exp(-z^2 / 2), for two values.
__device__ __forceinline__ float2 normal_tail2(float2 z) {
  const float2 d = fma2(both(0.311126984f), make_float2(fabsf(z.x), fabsf(z.y)), both(1.0f));
  const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
  float2 p = both(tail_coef(7));
#pragma unroll
  for (int k = 6; k >= 0; --k) p = fma2(p, t, both(tail_coef(k)));
  return mul2(p, t);
}

// Phi(z) from erfc(|z| / sqrt 2).
__device__ __forceinline__ float normal_cdf(float z, float h) { return z < 0.0f ? 0.5f * h : fmaf(-0.5f, h, 1.0f); }

// Two values at once, two operations to an instruction where there is one.
// Where 2^n overflows to infinity the reciprocal is 0, the limit.
template <int kAct>
__device__ __forceinline__ float2 act_value2(float2 z) {
  if constexpr (kAct == FALQON_ACT_RELU) return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);  // NaN stays
  if constexpr (kAct == FALQON_ACT_GELU_TANH || kAct == FALQON_ACT_SILU) {
    float2 n;
    if constexpr (kAct == FALQON_ACT_SILU)
      n = mul2(z, both(-kLog2E));
    else
      n = mul2(z, fma2(mul2(z, z), both(-kGeluTwoU * kLog2E * kGeluCubic), both(-kGeluTwoU * kLog2E)));
    const float2 d = add2(make_float2(exp2_fast(n.x), exp2_fast(n.y)), both(1.0f));
    return mul2(z, make_float2(rcp_fast(d.x), rcp_fast(d.y)));
  }
  if constexpr (kAct == FALQON_ACT_GELU_ERF) {
    const float2 q = mul2(mul2(z, z), both(-0.5f * kLog2E));
    const float2 h = mul2(normal_tail2(z), make_float2(exp2_fast(q.x), exp2_fast(q.y)));
    return mul2(z, make_float2(normal_cdf(z.x, h.x), normal_cdf(z.y, h.y)));
  }
  return z;
}

// Two derivatives at once.  With p = 1 / (1 + 2^n) the sigmoid forms are
// p + zu p (1 - p) = p (1 + zu (1 - p)); where 2^n overflows p is 0 and so is
// the product, as in the limit.
__device__ __forceinline__ float2 logistic_slope2(float2 n, float2 zu) {
  const float2 d = add2(make_float2(exp2_fast(n.x), exp2_fast(n.y)), both(1.0f));
  const float2 p = make_float2(rcp_fast(d.x), rcp_fast(d.y));
  return mul2(p, fma2(zu, fma2(p, both(-1.0f), both(1.0f)), both(1.0f)));
}

// Past some |z| a slope is 0 or 1 in float32 whatever z: z is held there, so
// that no product of the largest z overflows or meets a factor of 0 as an
// infinity.  The kept bf16 Z of a float32 bias of the lowest value, a mask, is
// -infinity; its slope is 0.  (NaN stays NaN.)
template <int kAct>
__device__ __forceinline__ float2 act_slope2(float2 z) {
  if constexpr (kAct == FALQON_ACT_RELU) return make_float2(z.x > 0.0f ? 1.0f : 0.0f, z.y > 0.0f ? 1.0f : 0.0f);
  if constexpr (kAct == FALQON_ACT_GELU_ERF) {
    z = clamp2(z, 20.0f);
    const float2 q = mul2(mul2(z, z), both(-0.5f * kLog2E));
    const float2 e = make_float2(exp2_fast(q.x), exp2_fast(q.y));
    const float2 h = mul2(normal_tail2(z), e);
    return fma2(mul2(z, both(kInvSqrt2Pi)), e, make_float2(normal_cdf(z.x, h.x), normal_cdf(z.y, h.y)));
  }
  if constexpr (kAct == FALQON_ACT_GELU_TANH) {
    z = clamp2(z, 20.0f);
    const float2 z2 = mul2(z, z);
    const float2 n = mul2(z, fma2(z2, both(-kGeluTwoU * kLog2E * kGeluCubic), both(-kGeluTwoU * kLog2E)));
    return logistic_slope2(n, mul2(z, fma2(z2, both(3.0f * kGeluTwoU * kGeluCubic), both(kGeluTwoU))));
  }
  if constexpr (kAct == FALQON_ACT_SILU) {
    z = clamp2(z, 100.0f);
    return logistic_slope2(mul2(z, both(-kLog2E)), z);
  }
  return both(1.0f);
}

}  // namespace falqon
