// activation.cuh -- the activations of the fused GEMM epilogues, on fp32 values, two at a time.
//
// exp2 and the reciprocal are the hardware approximations (2^-22 relative error each, documented by PTX), and the
// exponent s of 2^s is rounded to fp32, which is worth up to 2^-23 |s| of the exponential.  So an activation is within
// (|s| + 6) 2^-22 of its formula relative to the result: 2e-6 for |x| <= 1, at most 3.2e-5 at the end of the tail,
// |s| = 126, far below half a step of bf16 (2^-9).  Nothing is computed as 1 + tanh(x) or 1 + erf(x), which cancel for
// negative x.  Where 2^s is below the smallest normal number it is 0: a tail ends at magnitudes below 1.1e-36.
//
// Both run on the special-function unit, 4 lanes a clock in each SM quarter, and an epilogue that applies an
// activation is bound by it.  So two values share one reciprocal: 1/p = q / (pq), 1/q = p / (pq).
#pragma once

#include <cuda_runtime.h>

#include "bsp.h"

namespace bsp {

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

// max that keeps NaN.
__device__ __forceinline__ float max_nan(float x, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(c));
  return y;
}

// x / (1 + 2^-s) for both, s of x's sign, from t = 2^-|s| <= 1: x / (1 + t), and x t / (1 + t) where x < 0, so that
// nothing overflows and the tail of negative x is t's own, down to where t is below the smallest normal number (then
// -0).  The minimum takes nothing but a NaN, which must not reach the other value through the shared reciprocal: x
// itself keeps it.
__device__ __forceinline__ void logistic2(float& x0, float& x1, float s0, float s1) {
  const float t0 = fminf(ex2_approx(-fabsf(s0)), 1.0f), t1 = fminf(ex2_approx(-fabsf(s1)), 1.0f);
  const float p = 1.0f + t0, q = 1.0f + t1;
  const float r = rcp_approx(p * q);
  x0 *= (x0 < 0.0f ? t0 : 1.0f) * (r * q);
  x1 *= (x1 < 0.0f ? t1 : 1.0f) * (r * p);
}

// x / (1 + e^-x).  The maximum is for -infinity times a t of 0; at -1000 t has long been 0.
__device__ __forceinline__ void silu2(float& x0, float& x1) {
  x0 = max_nan(x0, -1000.0f);
  x1 = max_nan(x1, -1000.0f);
  logistic2(x0, x1, 1.44269504f * x0, 1.44269504f * x1);
}

// x/2 (1 + tanh u) = x / (1 + e^-2u), u = sqrt(2/pi) (x + 0.044715 x^3); the constants are 2 sqrt(2/pi) log2(e) and
// that times 0.044715.  The maximum as in silu2.
__device__ __forceinline__ void gelu_tanh2(float& x0, float& x1) {
  x0 = max_nan(x0, -1000.0f);
  x1 = max_nan(x1, -1000.0f);
  logistic2(x0, x1, x0 * fmaf(0.102943240f, x0 * x0, 2.30220820f), x1 * fmaf(0.102943240f, x1 * x1, 2.30220820f));
}

// x Phi(x) = max(x, 0) - |x| Q(|x|) with the normal tail Q(u) = e^(-u^2/2) P(1 / (1 + 0.23 u)).  P is a polynomial of
// degree 8 fitted to e^(u^2/2) Q(u) over 0 <= u <= 14 by iteratively reweighted least squares (largest relative
// error 4.8e-8; 6e-7 evaluated in fp32).  Beyond 14 the exponential is 0 in fp32; the clamp keeps |x| Q(|x|) at 0 for
// infinite x.
__device__ __forceinline__ float normal_tail(float u, float t) {
  float p = -0.0784672499f;
  p = fmaf(p, t, 0.290413111f);
  p = fmaf(p, t, -0.278124809f);
  p = fmaf(p, t, 0.30147028f);
  p = fmaf(p, t, -0.032918442f);
  p = fmaf(p, t, 0.119513303f);
  p = fmaf(p, t, 0.0857631117f);
  p = fmaf(p, t, 0.0923784301f);
  p = fmaf(p, t, -2.77608233e-05f);
  return ex2_approx(-0.72134752f * u * u) * p;
}

__device__ __forceinline__ void gelu2(float& x0, float& x1) {
  const float u0 = fminf(fabsf(x0), 32.0f), u1 = fminf(fabsf(x1), 32.0f);
  const float p = fmaf(0.23f, u0, 1.0f), q = fmaf(0.23f, u1, 1.0f);
  const float r = rcp_approx(p * q);
  x0 = fmaf(-u0, normal_tail(u0, r * q), max_nan(x0, 0.0f));
  x1 = fmaf(-u1, normal_tail(u1, r * p), max_nan(x1, 0.0f));
}

template <int ACT>
__device__ __forceinline__ void activate2(float& x0, float& x1) {
  if constexpr (ACT == BSP_ACT_RELU) {
    x0 = max_nan(x0, 0.0f);
    x1 = max_nan(x1, 0.0f);
  } else if constexpr (ACT == BSP_ACT_GELU) {
    gelu2(x0, x1);
  } else if constexpr (ACT == BSP_ACT_GELU_TANH) {
    gelu_tanh2(x0, x1);
  } else if constexpr (ACT == BSP_ACT_SILU) {
    silu2(x0, x1);
  }
}

}  // namespace bsp
