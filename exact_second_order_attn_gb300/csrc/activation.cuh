// Activations of a linear layer and their first two derivatives, in fp32.
//   relu       z > 0 ? z : 0 (a' = 0 at 0; a'' = 0)
//   gelu       z F(z), F the normal distribution's integral, f its density:
//              a' = F + z f, a'' = f (2 - z^2)
//   gelu_tanh  z s(v), s the logistic function, v = 2 sqrt(2 / pi) (z + 0.044715 z^3),
//              which is z (1 + tanh(v / 2)) / 2 without its cancellation at z < 0
//   silu       z s(z)
// (z s(v))' = s + z s' v', and (z s(v))'' = s' (2 v' + z v'' + z v'^2 (1 - 2 s)).
// s' = s(v) s(-v) is made of the exponential: s (1 - s) would lose it in the steps of s
// below 1 (gelu_tanh'' from z = 3 on, all of it at 5).
//
// EXACT (fp32 tensors) takes expf and erfcf.  For bf16 tensors, whose results are
// rounded to 2^-9, 2^x and 1/x of the special function unit (2^-22), and for erfc the
// form of Abramowitz and Stegun 7.1.26, exp(-x^2) times a polynomial of degree five in
// t = 1 / (1 + p x), two values in a packed instruction: the epilogues that call them
// are bound by issue.  Its coefficients are fitted here (p = 1/2; linear programme over
// 0 <= x <= 9.6): F(z) is within 2^-19.7, and within 2^-12 of itself for every z < 0 that
// bf16 holds.  Theirs, which are within 1.5e-7 but not relative to a small F, were off by
// 1.6e-3 of it at z = -5, 1 % at -8 and 3 % at -12, more than bf16's half step.
#pragma once

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "rowvec.cuh"

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
__device__ __forceinline__ float logistic(float v) {  // (the reciprocal is off by 2^-23 at most)
  return act_rcp(1.f + (EXACT ? expf(-v) : act_exp(-v)));
}

// erfc(x) / 2 = exp(-x^2) (kErfc1 t + ... + kErfc5 t^5), t = 1 / (1 + x / 2), x = |z| / sqrt(2).
constexpr float kErfcP = 0.5f * 0.70710678118654752f;
constexpr float kErfc1 = 0.5f * 0.27880181f, kErfc2 = 0.5f * 0.32172487f, kErfc3 = 0.5f * 0.07490349f,
                kErfc4 = 0.5f * 0.51318599f, kErfc5 = 0.5f * -0.18861556f;

// F(z), and f(z) sqrt(2 pi) = exp(-z^2 / 2).
template <bool EXACT>
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
  if (EXACT) {
    bell = expf(-0.5f * z * z);
    return 0.5f * erfcf(z * -0.70710678118654752f);
  }
  bell = act_exp(-0.5f * z * z);
  const float t = act_rcp(fmaf(fabsf(z), kErfcP, 1.f));
  float p = fmaf(kErfc5, t, kErfc4);
  p = fmaf(p, t, kErfc3);
  p = fmaf(p, t, kErfc2);
  p = fmaf(p, t, kErfc1);
  const float h = p * t * bell;
  return z > 0.f ? 1.f - h : h + 0.f * z;  // (0 z: a NaN stays one)
}

constexpr float kTanhC = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// The lesser of two values; a NaN stays one.
__device__ __forceinline__ float act_least(float z, float top) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(z) : "f"(top));
  return z;
}
// z moved into [-top, top]; a NaN stays one.
__device__ __forceinline__ float act_clamp(float z, float top) {
  z = act_least(z, top);
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

// --- eight values at a time, in packed pairs ----------------------------------------

using row::F2;

__device__ __forceinline__ F2 both(float f) { return row::pair(f, f); }
__device__ __forceinline__ F2 exp2_pair(F2 x) {
  const float2 f = row::parts(x);
  float a, b;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(f.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(f.y));
  return row::pair(a, b);
}
__device__ __forceinline__ F2 rcp_pair(F2 x) {
  const float2 f = row::parts(x);
  return row::pair(act_rcp(f.x), act_rcp(f.y));
}
// The logistic function of v, from -v log2(e).
__device__ __forceinline__ F2 logistic_pair(F2 x) { return rcp_pair(exp2_pair(x) + both(1.f)); }
// ... and its slope, u s^2 with u = 2^x, which stays finite (the slope is 0 long before).
__device__ __forceinline__ F2 logistic_pair(F2 x, F2& slope) {
  const float2 f = row::parts(x);
  const F2 u = exp2_pair(row::pair(act_least(f.x, 126.f), act_least(f.y, 126.f)));
  const F2 s = rcp_pair(u + both(1.f));
  slope = u * s * s;
  return s;
}
constexpr float kActLog2e = 1.4426950408889634f;

__device__ __forceinline__ F2 clamp_pair(F2 z, float top) {
  const float2 f = row::parts(z);
  return row::pair(act_clamp(f.x, top), act_clamp(f.y, top));
}

// As normal_cdf.
template <bool EXACT>
__device__ __forceinline__ F2 cdf_pair(F2 z, F2& bell) {
  if (EXACT) {
    const float2 f = row::parts(z);
    float a, b;
    const float x = normal_cdf<true>(f.x, a), y = normal_cdf<true>(f.y, b);
    bell = row::pair(a, b);
    return row::pair(x, y);
  }
  const F2 z2 = z * z;
  bell = exp2_pair(z2 * both(-0.5f * kActLog2e));
  const float2 f = row::parts(z);
  const F2 t = row::pair(act_rcp(fmaf(fabsf(f.x), kErfcP, 1.f)), act_rcp(fmaf(fabsf(f.y), kErfcP, 1.f)));
  F2 p = mad(t, both(kErfc5), both(kErfc4));
  p = mad(p, t, both(kErfc3));
  p = mad(p, t, both(kErfc2));
  p = mad(p, t, both(kErfc1));
  const F2 h = p * t * bell;
  const float2 lo = row::parts(h), hi = row::parts(mad(h, both(-1.f), both(1.f)));
  return row::pair(f.x > 0.f ? hi.x : lo.x, f.y > 0.f ? hi.y : lo.y);
}

template <int ACT>
__device__ __forceinline__ F2 value_pair(F2 z) {
  if (ACT == kActGelu) {
    F2 bell;
    return z * cdf_pair<false>(z, bell);
  }
  if (ACT == kActGeluTanh)
    return z * logistic_pair(z * mad(z * z, both(-0.044715f * kTanhC * kActLog2e), both(-kTanhC * kActLog2e)));
  return z * logistic_pair(z * both(-kActLog2e));  // kActSilu
}

// The logistic function of v and its slope; EXACT with expf.
template <bool EXACT>
__device__ __forceinline__ F2 logistic_of(F2 v, F2& slope) {
  if (!EXACT) return logistic_pair(v * both(-kActLog2e), slope);
  const float2 f = row::parts(v);
  const F2 e = row::pair(expf(-fabsf(f.x)), expf(-fabsf(f.y)));  // s(|v|) = 1 / (1 + e), s(-|v|) = e / (1 + e)
  const F2 hi = rcp_pair(e + both(1.f)), lo = e * hi;
  slope = lo * hi;
  const float2 a = row::parts(hi), b = row::parts(lo);
  return row::pair(f.x < 0.f ? b.x : a.x, f.y < 0.f ? b.y : a.y);
}

// a' (and, SECOND, a'').  (Not EXACT: z was kept in fp16, no power of it overflows.)
template <int ACT, bool EXACT, bool SECOND>
__device__ __forceinline__ F2 slope_pair(F2 z, F2& curve) {
  const F2 c = EXACT ? clamp_pair(z, ACT == kActSilu ? kSiluTop : kActTop) : z;
  if (ACT == kActGelu) {
    F2 bell;
    const F2 up = cdf_pair<EXACT>(c, bell), f = bell * both(0.39894228040143268f);
    if (SECOND) curve = f * mad(c * c, both(-1.f), both(2.f));
    return mad(c, f, up);
  }
  if (ACT == kActGeluTanh) {
    const F2 c2 = c * c;
    F2 d;
    const F2 s = EXACT ? logistic_of<true>(c * mad(c2, both(0.044715f * kTanhC), both(kTanhC)), d)
                       : logistic_pair(c * mad(c2, both(-0.044715f * kTanhC * kActLog2e), both(-kTanhC * kActLog2e)), d);
    const F2 v1 = mad(c2, both(3.f * 0.044715f * kTanhC), both(kTanhC)), zv = c * v1;
    if (SECOND)  // 2 v' + z v'' = 4 v' - 4 sqrt(2 / pi)
      curve = d * mad(zv, v1 * mad(s, both(-2.f), both(1.f)), mad(v1, both(4.f), both(-2.f * kTanhC)));
    return mad(zv, d, s);
  }
  // kActSilu
  F2 d;
  const F2 s = logistic_of<EXACT>(c, d);
  if (SECOND) curve = d * mad(c, mad(s, both(-2.f), both(1.f)), both(2.f));
  return mad(c, d, s);
}

// a[j] *= b[j], a[j] += b[j].
__device__ __forceinline__ void mul8(float* a, const float* b) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 f = row::parts(row::pair(a[j], a[j + 1]) * row::pair(b[j], b[j + 1]));
    a[j] = f.x, a[j + 1] = f.y;
  }
}
__device__ __forceinline__ void add8(float* a, const float* b) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 f = row::parts(row::pair(a[j], a[j + 1]) + row::pair(b[j], b[j + 1]));
    a[j] = f.x, a[j + 1] = f.y;
  }
}

template <int ACT>
constexpr bool kSmooth = ACT == kActGelu || ACT == kActGeluTanh || ACT == kActSilu;

// z[j] becomes a(z[j]).
template <int ACT, bool EXACT>
__device__ __forceinline__ void act_values8(float* z) {
  if constexpr (!EXACT && kSmooth<ACT>) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 f = row::parts(value_pair<ACT>(row::pair(z[j], z[j + 1])));
      z[j] = f.x, z[j + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = act_value<ACT, EXACT>(z[j]);
  }
}
// z[j] becomes a'(z[j]), and (SECOND) a2[j] a''.
template <int ACT, bool EXACT, bool SECOND>
__device__ __forceinline__ void act_slopes8(float* z, float* a2) {
  if constexpr (kSmooth<ACT>) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      F2 c;
      const float2 f = row::parts(slope_pair<ACT, EXACT, SECOND>(row::pair(z[j], z[j + 1]), c));
      z[j] = f.x, z[j + 1] = f.y;
      if (SECOND) {
        const float2 g = row::parts(c);
        a2[j] = g.x, a2[j + 1] = g.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] = ACT == kActRelu && z[j] <= 0.f ? 0.f : 1.f;
      if (SECOND) a2[j] = 0.f;
    }
  }
}

// The same with the activation as a value.
template <bool EXACT>
__device__ __forceinline__ void act_values8(int act, float* z) {
  switch (act) {
    case kActRelu: return act_values8<kActRelu, EXACT>(z);
    case kActGelu: return act_values8<kActGelu, EXACT>(z);
    case kActGeluTanh: return act_values8<kActGeluTanh, EXACT>(z);
    case kActSilu: return act_values8<kActSilu, EXACT>(z);
    default: return;
  }
}
template <bool EXACT>
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case kActRelu: return act_value<kActRelu, EXACT>(z);
    case kActGelu: return act_value<kActGelu, EXACT>(z);
    case kActGeluTanh: return act_value<kActGeluTanh, EXACT>(z);
    case kActSilu: return act_value<kActSilu, EXACT>(z);
    default: return z;
  }
}
template <bool EXACT>
__device__ __forceinline__ void act_slopes8(int act, float* z) {
  switch (act) {
    case kActRelu: return act_slopes8<kActRelu, EXACT, false>(z, nullptr);
    case kActGelu: return act_slopes8<kActGelu, EXACT, false>(z, nullptr);
    case kActGeluTanh: return act_slopes8<kActGeluTanh, EXACT, false>(z, nullptr);
    case kActSilu: return act_slopes8<kActSilu, EXACT, false>(z, nullptr);
    default:
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = 1.f;
  }
}

}  // namespace fbob
