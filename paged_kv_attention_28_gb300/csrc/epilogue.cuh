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

// gelu_tanh(y) = y/2 (1 + tanh u) = y sigmoid(2u), u = sqrt(2/pi) (y + 0.044715 y^3), and silu(y) =
// y sigmoid(y): both as y / (1 + 2^t), which keeps the relative precision of small results.
// erff is off by 2 units in the last place of 1, i.e. 2^-23 |y| here.
template <int ACT>
__device__ __forceinline__ float activate(float y) {
  if constexpr (ACT == PKV_ACT_RELU) {  // NaN stays
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(y));
    return r;
  }
  if constexpr (ACT == PKV_ACT_GELU) return 0.5f * y * (1.0f + erff(y * 0.70710678118654752f));
  if constexpr (ACT == PKV_ACT_GELU_TANH) {
    const float t = y * fmaf(y * y, -2.0f * 1.4426950408889634f * 0.7978845608028654f * 0.044715f,
                             -2.0f * 1.4426950408889634f * 0.7978845608028654f);
    return __fdividef(y, 1.0f + ex2(t));
  }
  if constexpr (ACT == PKV_ACT_SILU) return __fdividef(y, 1.0f + ex2(-1.4426950408889634f * y));
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
