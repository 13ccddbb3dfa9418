// Activations of a linear layer and their first two derivatives, in fp32.
//   relu       z > 0 ? z : 0 (a' = 0 at 0; a'' = 0)
//   gelu       z F(z), F the normal distribution's integral, f its density:
//              a' = F + z f, a'' = f (2 - z^2)
//   gelu_tanh  z s(v), s the logistic function, v = 2 sqrt(2 / pi) (z + 0.044715 z^3),
//              which is z (1 + tanh(v / 2)) / 2 without its cancellation at z < 0
//   silu       z s(z)
// With s' = s (1 - s): (z s(v))' = s + z s' v', and
// (z s(v))'' = s' (2 v' + z v'' + z v'^2 (1 - 2 s)).
//
// EXACT (fp32 tensors) takes expf and erfcf.  For bf16 tensors, whose results are
// rounded to 2^-9, 2^x and 1/x of the special function unit (2^-22), and
// Abramowitz and Stegun 7.1.26 for erfc (1.5e-7; relative to F 2e-4 at z = -4,
// 2e-3 at z = -5): the epilogues that call them are bound by issue.
#pragma once

#include <math.h>
#include <stdint.h>

#include "internal.h"

namespace fbob {

__device__ __forceinline__ float act_exp(float x) {  // fast e^x
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float act_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool EXACT>
__device__ __forceinline__ float logistic(float v) {
  return EXACT ? 1.f / (1.f + expf(-v)) : act_rcp(1.f + act_exp(-v));
}

// F(z), and f(z) sqrt(2 pi) = exp(-z^2 / 2).
template <bool EXACT>
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  if (EXACT) {
    bell = expf(-0.5f * z * z);
    return 0.5f * erfcf(z * -0.70710678118654752f);
  }
  bell = act_exp(-0.5f * z * z);
  const float x = fabsf(z) * 0.70710678118654752f, t = act_rcp(fmaf(0.3275911f, x, 1.f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float h = 0.5f * p * t * bell;
  return z > 0.f ? 1.f - h : h + 0.f * z;  // (0 z: a NaN stays one)
}

constexpr float kTanhC = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// z moved into [-top, top]; a NaN stays one.
__device__ __forceinline__ float act_clamp(float z, float top) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(z) : "f"(top));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(z) : "f"(-top));
  return z;
}
// Beyond these s' and f are 0, and squares of what lies further out would overflow
// into 0 inf.
constexpr float kActTop = 32.f, kSiluTop = 128.f;

template <int ACT, bool EXACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == kActRelu) return z <= 0.f ? 0.f : z;
  if (ACT == kActGelu) {
    float bell;
    return z * normal_cdf<EXACT>(z, bell);
  }
  if (ACT == kActGeluTanh) {
    // (no clamp: where z^3 overflows s is 0 or 1)
    return z * logistic<EXACT>(z * fmaf(0.044715f * kTanhC * z, z, kTanhC));
  }
  if (ACT == kActSilu) return z * logistic<EXACT>(z);
  return z;
}

// a' (and, SECOND, a'').
template <int ACT, bool EXACT, bool SECOND>
__device__ __forceinline__ float act_slope(float z, float& curve) {
  if (ACT == kActRelu) {
    curve = 0.f;
    return z <= 0.f ? 0.f : 1.f;
  }
  if (ACT == kActGelu) {
    const float c = act_clamp(z, kActTop);
    float bell;
    const float up = normal_cdf<EXACT>(c, bell), f = 0.39894228040143268f * bell;
    if (SECOND) curve = f * fmaf(-c, c, 2.f);
    return fmaf(c, f, up);
  }
  if (ACT == kActGeluTanh) {
    const float c = act_clamp(z, kActTop), c2 = 0.044715f * c * c;
    const float s = logistic<EXACT>(kTanhC * fmaf(c2, c, c)), d = s * (1.f - s);
    const float v1 = kTanhC * fmaf(3.f, c2, 1.f), zv = c * v1;
    if (SECOND) curve = d * fmaf(zv, v1 * fmaf(-2.f, s, 1.f), fmaf(2.f, v1, kTanhC * 6.f * c2));
    return fmaf(zv, d, s);
  }
  if (ACT == kActSilu) {
    const float c = act_clamp(z, kSiluTop);
    const float s = logistic<EXACT>(c), d = s * (1.f - s);
    if (SECOND) curve = d * fmaf(c, fmaf(-2.f, s, 1.f), 2.f);
    return fmaf(c, d, s);
  }
  curve = 0.f;
  return 1.f;
}

// a(z) of n values.
template <bool EXACT, int N>
__device__ __forceinline__ void act_values(int act, float* z) {
#define FBOB_ACT_CASE(A)                                                 \
  case A:                                                                \
    _Pragma("unroll") for (int j = 0; j < N; ++j) z[j] = act_value<A, EXACT>(z[j]); \
    break;
  switch (act) {
    FBOB_ACT_CASE(kActRelu)
    FBOB_ACT_CASE(kActGelu)
    FBOB_ACT_CASE(kActGeluTanh)
    FBOB_ACT_CASE(kActSilu)
    default: break;
  }
#undef FBOB_ACT_CASE
}

// z[j] becomes a'(z[j]) of n values, a2[j] a''(z[j]).
template <bool EXACT, bool SECOND, int N>
__device__ __forceinline__ void act_slopes(int act, float* z, float* a2) {
  float none;
#define FBOB_ACT_CASE(A)                                                              \
  case A:                                                                             \
    _Pragma("unroll") for (int j = 0; j < N; ++j) z[j] =                              \
        act_slope<A, EXACT, SECOND>(z[j], SECOND ? a2[j] : none);                     \
    break;
  switch (act) {
    FBOB_ACT_CASE(kActRelu)
    FBOB_ACT_CASE(kActGelu)
    FBOB_ACT_CASE(kActGeluTanh)
    FBOB_ACT_CASE(kActSilu)
    default:
#pragma unroll
      for (int j = 0; j < N; ++j) {
        z[j] = 1.f;
        if (SECOND) a2[j] = 0.f;
      }
      break;
  }
#undef FBOB_ACT_CASE
}

}  // namespace fbob
