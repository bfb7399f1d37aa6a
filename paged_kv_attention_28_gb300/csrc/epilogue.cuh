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
// The quotient for every y is 1 % faster (2611 x 11008 x 256 with silu 35.3 for 35.6 us); one value at a time 4 % slower.
__device__ __forceinline__ void over_one_plus_exp4(float& y0, float& y1, Two t) {
  float t0, t1, d0, d1, s0, s1;
  split(t, t0, t1);
  const Two y = two(y0, y1), h = two(ex2(-fabsf(t0)), ex2(-fabsf(t1)));
  split(fma2(h, h, two(1.0f, 1.0f)), d0, d1);
  split(mul2(mul2(y, h), h), s0, s1);
  split(mul2(two(t0 > 0.0f ? s0 : y0, t1 > 0.0f ? s1 : y1), two(rcp(d0), rcp(d1))), y0, y1);
}

// gelu(y) = y Phi(y), Phi the normal distribution. With a = |y| and q = Phi(-a) it is y q below 0 and y (1 - q) above:
// no difference of nearly equal numbers, where 1 + erf loses all of a result below -5 (its error is
// 2^-23 |y|, the result -1.4e-6). q = P(s) h^2 with h = exp(-a^2 / 4), s = 1 / (1 + 0.3 a); P is the polynomial of
// degree 8 that is nearest to Phi(-a) exp(a^2 / 2) for 0 <= a <= 14.5 (a weighted least-squares fit on Chebyshev
// nodes of s, reweighted until its relative errors are even: 6e-8). In fp32 the result is off by
// 2^-22 |y| and by 2^-17 of itself, more only below fp32's smallest normal number. 2611 x 11008 x 256: 61 us with
// erff, 47 with this, 48 where it takes two values at a time.
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
// y sigmoid(y), the sigmoids as 1 / (1 + 2^(2 t)).
template <int ACT>
__device__ __forceinline__ void activate(float& y0, float& y1) {
  constexpr float kL = 1.4426950408889634f, kU = kL * 0.7978845608028654f;  // log2 e, and times sqrt(2/pi)
  if constexpr (ACT == PKV_ACT_RELU) {  // NaN stays
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(y0));
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(y1));
  } else if constexpr (ACT == PKV_ACT_GELU) {
    y0 = gelu(y0);
    y1 = gelu(y1);
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
