// What a matrix product's accumulator goes through before it is stored: bias, activation,
// residual, one rounding to bf16.
#pragma once

#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {

struct Epilogue {
  const __nv_bfloat16* bias;      // [n] or null
  const __nv_bfloat16* residual;  // [m][n] or null
  int activation;
};

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// gelu(y) = y Phi(y), Phi the normal distribution. With a = |y| and q = Phi(-a) it is y q below 0 and y (1 - q) above:
// no difference of nearly equal numbers, where 1 + erf loses all of a result below -5 (its error is
// 2^-23 |y|, the result -1.4e-6). q = P(s) h^2 with h = exp(-a^2 / 4), s = 1 / (1 + 0.3 a); P is the polynomial of
// degree 8 that is nearest to Phi(-a) exp(a^2 / 2) for 0 <= a <= 14.5 (a weighted least-squares fit on Chebyshev
// nodes of s, reweighted until its relative errors are even: 6e-8). In fp32 the result is off by
// 2^-22 |y| and by 2^-17 of itself, more only below fp32's smallest normal number. 2611 x 11008 x 256: 61 us with
// erff, 49 with this.
__device__ __forceinline__ float gelu(float y) {
  constexpr float kP[9] = {0x1.eec024p-18f, 0x1.e96848p-4f, 0x1.f37ce0p-4f, 0x1.836c7ep-4f, 0x1.246216p-3f,
                           -0x1.3abc1cp-4f, 0x1.d4e49cp-3f, -0x1.5abddap-3f, 0x1.3aa222p-5f};
  const float s = rcp(fmaf(fabsf(y), 0.3f, 1.0f)), h = ex2(y * (-0.25f * 1.4426950408889634f) * y);
  float p = kP[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) p = fmaf(p, s, kP[i]);
  const float q = p * h * h;
  return y * (y > 0.0f ? 1.0f - q : q);
}

// gelu_tanh(y) = y/2 (1 + tanh u) = y sigmoid(2u), u = sqrt(2/pi) (y + 0.044715 y^3), and silu(y) =
// y sigmoid(y). sigmoid = 1 / (1 + 2^t) keeps the relative precision of small results, but a reciprocal of a number
// past 2^126 comes back as 0, which for silu is at y = -87.3, where the result is still 1e-36. With the
// divisor scaled by 2^-16 that is at t = 142, past bf16's smallest numbers. 4096 x 11008 x 4096 takes the same time
// as with y / (1 + 2^t), 2611 x 11008 x 256 with silu 35.9 us for 35.0.
__device__ __forceinline__ float times_sigmoid(float y, float t16) {  // t - 16
  return y * (rcp(ex2(t16) + 0x1p-16f) * 0x1p-16f);
}

template <int ACT>
__device__ __forceinline__ float activate(float y) {
  if constexpr (ACT == PKV_ACT_RELU) {  // NaN stays
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(y));
    return r;
  }
  constexpr float kL = 1.4426950408889634f, kU = kL * 2.0f * 0.7978845608028654f;  // log2 e, and times 2 sqrt(2/pi)
  if constexpr (ACT == PKV_ACT_GELU) return gelu(y);
  if constexpr (ACT == PKV_ACT_GELU_TANH)
    return times_sigmoid(y, fmaf(y, fmaf(y * y, -kU * 0.044715f, -kU), -16.0f));
  if constexpr (ACT == PKV_ACT_SILU) return times_sigmoid(y, fmaf(y, -kL, -16.0f));
  return y;
}

// y[i] = act(y[i]) for N values; the choice is uniform, so it is made once per call.
template <int N>
__device__ __forceinline__ void activate_all(float (&y)[N], int act) {
#define PKV_ACT_CASE(A)                                    \
  case A: {                                                \
    _Pragma("unroll") for (int i = 0; i < N; ++i) y[i] = activate<A>(y[i]); \
    break;                                                 \
  }
  switch (act) {
    PKV_ACT_CASE(PKV_ACT_RELU)
    PKV_ACT_CASE(PKV_ACT_GELU)
    PKV_ACT_CASE(PKV_ACT_GELU_TANH)
    PKV_ACT_CASE(PKV_ACT_SILU)
    default: break;
  }
#undef PKV_ACT_CASE
}

}  // namespace pkv
