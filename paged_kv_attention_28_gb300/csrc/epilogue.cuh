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

// Two fp32 values in a register pair, for the two-wide multiplies and fused multiply-adds.
using Two = uint64_t;
__device__ __forceinline__ Two two(float x, float y) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void split(Two v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// y / (1 + 2^(2 t)) for two values, with h = 2^-|t|: y / (1 + h^2) for t <= 0 and y h^2 / (1 + h^2) above, which keeps
// the relative precision of small results. (A quotient by a divisor past 2^126 comes back as 0, which for
// silu is at y = -87.3, where the result is still 1e-36.) h stays a normal number where h^2 is none.
// Against one value at a time and the quotient: 2611 x 11008 x 256 35.3 to 36.2 us with silu, 37.0 to 36.8 with
// gelu_tanh.
__device__ __forceinline__ void over_one_plus_exp4(float& y0, float& y1, Two t) {
  float t0, t1, d0, d1, s0, s1;
  split(t, t0, t1);
  const Two y = two(y0, y1), h = two(ex2(-fabsf(t0)), ex2(-fabsf(t1)));
  split(fma2(h, h, two(1.0f, 1.0f)), d0, d1);
  split(mul2(mul2(y, h), h), s0, s1);
  split(mul2(two(t0 > 0.0f ? s0 : y0, t1 > 0.0f ? s1 : y1), two(rcp(d0), rcp(d1))), y0, y1);
}

// gelu_tanh(y) = y/2 (1 + tanh u) = y sigmoid(2u), u = sqrt(2/pi) (y + 0.044715 y^3), and silu(y) =
// y sigmoid(y), the sigmoids as 1 / (1 + 2^(2 t)).
// erff is off by 2 units in the last place of 1, i.e. 2^-23 |y| here.
template <int ACT>
__device__ __forceinline__ void activate(float& y0, float& y1) {
  constexpr float kL = 1.4426950408889634f, kU = kL * 0.7978845608028654f;  // log2 e, and times sqrt(2/pi)
  if constexpr (ACT == PKV_ACT_RELU) {  // NaN stays
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(y0));
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(y1));
  } else if constexpr (ACT == PKV_ACT_GELU) {
    y0 = 0.5f * y0 * (1.0f + erff(y0 * 0.70710678118654752f));
    y1 = 0.5f * y1 * (1.0f + erff(y1 * 0.70710678118654752f));
  } else if constexpr (ACT == PKV_ACT_GELU_TANH) {
    const Two y = two(y0, y1);
    over_one_plus_exp4(y0, y1, mul2(y, fma2(mul2(y, y), two(-kU * 0.044715f, -kU * 0.044715f), two(-kU, -kU))));
  } else if constexpr (ACT == PKV_ACT_SILU) {
    over_one_plus_exp4(y0, y1, mul2(two(y0, y1), two(-0.5f * kL, -0.5f * kL)));
  }
}

// y[i] = act(y[i]) for N values; the choice is uniform, so it is made once per call.
template <int N>
__device__ __forceinline__ void activate_all(float (&y)[N], int act) {
  static_assert(N % 2 == 0, "pairs");
#define PKV_ACT_CASE(A)                                                                    \
  case A: {                                                                                \
    _Pragma("unroll") for (int i = 0; i < N; i += 2) activate<A>(y[i], y[i + 1]);          \
    break;                                                                                 \
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
