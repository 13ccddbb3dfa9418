// Vectors of a row as they lie in memory (16 bytes, or one element where rows
// or pointers are not 16-byte aligned), read as fp32 and written with one
// rounding.  Used by the row-wise kernels (layer norm, rotary positions).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace fbob {
namespace row {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// VEC elements of type T, kept in registers in the memory format (a bf16
// vector takes half the registers of its fp32 values).
template <typename T, int VEC>
struct Raw;

template <>
struct Raw<bf16, 8> {
  uint32_t u[4];
  __device__ __forceinline__ void load(const bf16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
  }
  __device__ __forceinline__ void store(bf16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? (u[i >> 1] & 0xffff0000u) : (u[i >> 1] << 16));
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
};

template <>
struct Raw<bf16, 1> {
  bf16 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *p; }
  __device__ __forceinline__ void store(bf16* p) const { *p = v; }
  __device__ __forceinline__ float get(int) const { return __bfloat162float(v); }
  __device__ __forceinline__ void set(const float* f) { v = __float2bfloat16_rn(f[0]); }
};

template <>
struct Raw<float, 4> {
  float v[4];
  __device__ __forceinline__ void load(const float* p) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f[i];
  }
};

template <>
struct Raw<float, 8> {
  Raw<float, 4> a, b;
  __device__ __forceinline__ void load(const float* p) { a.load(p), b.load(p + 4); }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a.v[i & 3] : b.v[i & 3]; }
};

template <>
struct Raw<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void store(float* p) const { *p = v; }
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void set(const float* f) { v = f[0]; }
};

// Elements of T in 16 bytes.
template <typename T>
constexpr int kFull = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ T from_float(float f);
template <>
__device__ __forceinline__ float from_float<float>(float f) { return f; }
template <>
__device__ __forceinline__ bf16 from_float<bf16>(float f) { return __float2bfloat16_rn(f); }

}  // namespace row
}  // namespace fbob
