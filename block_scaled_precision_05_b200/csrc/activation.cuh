// activation.cuh -- the activations of the fused GEMM epilogues, on fp32 values.
//
// exp2 and the reciprocal are the hardware approximations (2^-22 relative error each, documented by PTX), so an
// activation is within about 1e-6 of its formula relative to the result, far below half a step of bf16 (2^-9), and
// below the rounding noise of an fp32 sum over K.  Tails keep their relative accuracy: nothing is computed as
// 1 + tanh(x) or 1 + erf(x), which cancel for negative x.
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

// max(x, 0) that keeps NaN.
__device__ __forceinline__ float act_relu(float x) { return x < 0.0f ? 0.0f : x; }

// x / (1 + e^-x).
__device__ __forceinline__ float act_silu(float x) {
  return x * rcp_approx(1.0f + ex2_approx(-1.44269504f * x));
}

// x/2 (1 + tanh u) = x / (1 + e^-2u), u = sqrt(2/pi) (x + 0.044715 x^3); the constants are 2 sqrt(2/pi) log2(e) and
// that times 0.044715.
__device__ __forceinline__ float act_gelu_tanh(float x) {
  const float s = x * fmaf(0.102943240f, x * x, 2.30220820f);
  return x * rcp_approx(1.0f + ex2_approx(-s));
}

// x Phi(x) = max(x, 0) - |x| Q(|x|) with the normal tail Q(u) = e^(-u^2/2) P(1 / (1 + 0.23 u)).  P is a polynomial of
// degree 8 fitted to e^(u^2/2) Q(u) over 0 <= u <= 14 by iteratively reweighted least squares (largest relative
// error 4.8e-8; 6e-7 evaluated in fp32).  Beyond 14 the exponential is 0 in fp32; the clamp keeps |x| Q(|x|) at 0 for
// infinite x.
__device__ __forceinline__ float act_gelu(float x) {
  const float u = fminf(fabsf(x), 32.0f);
  const float t = rcp_approx(fmaf(0.23f, u, 1.0f));
  float p = -0.0784672499f;
  p = fmaf(p, t, 0.290413111f);
  p = fmaf(p, t, -0.278124809f);
  p = fmaf(p, t, 0.30147028f);
  p = fmaf(p, t, -0.032918442f);
  p = fmaf(p, t, 0.119513303f);
  p = fmaf(p, t, 0.0857631117f);
  p = fmaf(p, t, 0.0923784301f);
  p = fmaf(p, t, -2.77608233e-05f);
  return fmaf(-u * ex2_approx(-0.72134752f * u * u), p, act_relu(x));
}

template <int ACT>
__device__ __forceinline__ float activate(float y) {
  if constexpr (ACT == BSP_ACT_RELU) return act_relu(y);
  else if constexpr (ACT == BSP_ACT_GELU) return act_gelu(y);
  else if constexpr (ACT == BSP_ACT_GELU_TANH) return act_gelu_tanh(y);
  else if constexpr (ACT == BSP_ACT_SILU) return act_silu(y);
  else return y;
}

}  // namespace bsp
