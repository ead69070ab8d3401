// The gate of a gated feed-forward block, act(a) = a logistic(v(a)) with
// v = a (SiLU) or v = 2 sqrt(2/pi) (a + 0.044715 a^3) (GELU in its tanh form:
// (1 + tanh z) / 2 = logistic(2 z)).
#pragma once

#include "device.hpp"

namespace fp8bs {

// 1 / (1 + exp(-v)) by the hardware's exp2 and reciprocal (1 ulp each).  The
// product -v log2(e) carries its rounding error along (it would grow to v
// rounding steps in the exponential): within 2^-22 of the value for v > -87, and
// 0 below -89; infinities and NaN act as in the formula.
__device__ __forceinline__ float logistic(float v) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147181f;
  const float t = -v * kLog2e;
  const float rest = __builtin_fmaf(-v, kLog2eRest, __builtin_fmaf(-v, kLog2e, -t));
  float e = __builtin_amdgcn_exp2f(t);
  if (fabsf(t) < 126.0f) e = __builtin_fmaf(e * kLn2, rest, e);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

constexpr float kGeluA = 1.59576912f, kGeluB = 0.0713548163f;   // 2 sqrt(2/pi), and 0.044715 times it
__device__ __forceinline__ float gelu_argument(float a) { return a * __builtin_fmaf(kGeluB, a * a, kGeluA); }
// finite for every finite a (it meets a factor that is 0 far out)
__device__ __forceinline__ float gelu_argument_slope(float a) { return __builtin_fmaf(3.0f * kGeluB, fminf(a * a, 1e30f), kGeluA); }

}  // namespace fp8bs
