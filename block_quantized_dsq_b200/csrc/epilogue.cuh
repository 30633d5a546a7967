// epilogue.cuh -- what a fused product does with its fp32 sums before they
// leave the chip: y = act(v0 + bias0) [* (v1 + bias1)] + residual, each step
// one fp32 operation.
#pragma once

#include <cuda_runtime.h>

#include "../../include/dsq.h"

namespace dsq {

inline bool valid_act(int act) { return act >= DSQ_ACT_NONE && act <= DSQ_ACT_RELU; }

#ifdef __CUDACC__
// The activations keep their relative accuracy on the side where they vanish:
// every exponential has a negative argument (no overflow), and no step cancels.
// Errors below are relative, in units of 2^-24; where the factor on v is below
// 2^-126 it has fewer bits or may be 0.

// 1 / y for y >= 1 (the plain instruction, without the scaling that __fdividef
// adds for y beyond 2^126, where this is 0).
__device__ __forceinline__ float quick_rcp(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// 1 / (1 + exp(-w)): CUDA's expf is within 4, the reciprocal within 2.
__device__ __forceinline__ float sigmoid(float w) {
  const float e = expf(-fabsf(w));
  return (w < 0.0f ? e : 1.0f) * quick_rcp(1.0f + e);
}

// v * Phi(v).  Phi(-x) = exp(-x^2 / 2) g(x) for x >= 0, where g falls from 1/2 like
// 1 / x: t Q(t) with t = 1 / (1 + 0.3 x) and Q of degree 7, fitted here for equal
// relative ripples over 0 <= x <= 14.6 (within 3), where exp(-x^2 / 2) reaches 0.
// On the other side Phi is 1 less that.  All steps together: at most 37 + v^2 / 2,
// the latter from the rounded square; 11 + v^2 / 2 found.  An approximation of erf
// itself (1.5e-7 absolute) is 5e-4 off at v = -4; CUDA's erfcf takes several times as long.
__device__ __forceinline__ float gelu_erf(float v) {
  const float x = fabsf(v);
  const float t = quick_rcp(fmaf(0.3f, x, 1.0f));
  float q = fmaf(0.035374183f, t, -0.15595266f);
  q = fmaf(q, t, 0.20420371f);
  q = fmaf(q, t, -0.05171087f);
  q = fmaf(q, t, 0.12752204f);
  q = fmaf(q, t, 0.10022692f);
  q = fmaf(q, t, 0.12070406f);
  q = fmaf(q, t, 0.11963253f);
  const float c = q * t * expf(-(0.5f * x) * x);   // Phi(-x)
  return v * (v < 0.0f ? c : 1.0f - c);
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case DSQ_ACT_SILU: return v * sigmoid(v);   // at most 9
    case DSQ_ACT_GELU: return gelu_erf(v);
    // (1 + tanh u) / 2 = sigmoid(2u), 2u = 2 sqrt(2 / pi) (v + 0.044715 v^3): at most
    // 9 + 4 |2u|, where 1 + tanh would cancel
    case DSQ_ACT_GELU_TANH: return v * sigmoid(v * fmaf(0.071354814f * v, v, 1.59576912f));
    case DSQ_ACT_RELU: return v < 0.0f ? 0.0f : v;   // a NaN stays
    default: return v;
  }
}
#endif

}  // namespace dsq
