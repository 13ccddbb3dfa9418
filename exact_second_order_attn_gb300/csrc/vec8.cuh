// Eight neighbouring elements of a row as fp32, in 16-byte accesses (VEC: the
// caller has checked addresses and that all eight are there) or one by one, `n` of
// them at most.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace fbob {

// How z of a linear layer is kept: fp32, or fp16 beside bf16 tensors - eleven bits
// where bf16 has eight, and no activation's slope changes above its range (which is
// kept in by clamping; a NaN stays one).  Below 2^-25 it rounds to 0, where the smooth slopes
// are what they are at 0, but relu's is not that of a positive z: those are kept as
// 2^-24 at least.
template <typename T>
using Kept = std::conditional_t<sizeof(T) == 2, __half, float>;
__device__ __forceinline__ float kept_range(float z) { return z > 65504.f ? 65504.f : z < -65504.f ? -65504.f : z; }
__device__ __forceinline__ float kept_sign(float z) { return z > 0.f ? fmaxf(z, 0x1p-24f) : z; }

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  uint32_t h;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
  return h;
}
__device__ __forceinline__ void half8(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    v[2 * j] = f.x, v[2 * j + 1] = f.y;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float* v) {
  if constexpr (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? (float)p[j] : 0.f;
  } else if constexpr (std::is_same_v<T, __half>) {
    half8(*reinterpret_cast<const uint4*>(p), v);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const float4 f = *reinterpret_cast<const float4*>(p), g = *reinterpret_cast<const float4*>(p + 4);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w, v[4] = g.x, v[5] = g.y, v[6] = g.z, v[7] = g.w;
  }
}

// Eight elements as they came, so that more of them can be on their way.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) == 2 ? 1 : 2];
  template <bool VEC>
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)(sizeof(w) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = j < n ? p[j] : T(0.f);
    }
  }
  __device__ __forceinline__ void values(float* v) const {
    if constexpr (sizeof(T) == 4) {
      const float* f = reinterpret_cast<const float*>(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = f[j];
    } else if constexpr (std::is_same_v<T, __half>) {
      half8(w[0], v);
    } else {
      const uint32_t h[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(h[j] << 16);
        v[2 * j + 1] = __uint_as_float(h[j] & 0xffff0000u);
      }
    }
  }
};

// Eight values as bf16 pairs.
__device__ __forceinline__ uint4 bf16x8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
  if constexpr (!VEC) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n) p[j] = (T)(std::is_same_v<T, __half> ? kept_range(v[j]) : v[j]);
    }
  } else if constexpr (std::is_same_v<T, __half>) {
    *reinterpret_cast<uint4*>(p) = make_uint4(half_pair(v[0], v[1]), half_pair(v[2], v[3]), half_pair(v[4], v[5]),
                                              half_pair(v[6], v[7]));
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = bf16x8(v);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace fbob
