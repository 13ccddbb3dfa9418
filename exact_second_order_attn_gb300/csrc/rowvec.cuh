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

// Two fp32 values in a register pair: one packed instruction does both.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 parts(F2 a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
  return f;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mad(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float mad(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(F2 a) {
  const float2 f = parts(a);
  return f.x + f.y;
}
__device__ __forceinline__ float total(float a) { return a; }

// The unit of arithmetic on vectors of VEC elements: pairs, or single values.
template <int VEC>
struct UnitOf {
  using type = F2;
};
template <>
struct UnitOf<1> {
  using type = float;
};
template <int VEC>
using Unit = typename UnitOf<VEC>::type;
template <int VEC>
constexpr int kUnits = VEC > 1 ? VEC / 2 : 1;
__device__ __forceinline__ void fill(F2& u, float f) { u = pair(f, f); }
__device__ __forceinline__ void fill(float& u, float f) { u = f; }
template <int VEC>
__device__ __forceinline__ Unit<VEC> all(float f) {
  Unit<VEC> u;
  fill(u, f);
  return u;
}

// VEC elements of type T, kept in registers in the memory format (a bf16
// vector takes half the registers of its fp32 values).  unit(i) gives the
// values of unit i, put(i) rounds them back; renew() hides the values' origin
// from the compiler, so that fp32 expansions made before it are made again
// after it instead of being held in registers in between.
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
  __device__ __forceinline__ F2 unit(int i) const {
    return pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void put(int i, F2 x) {
    const float2 f = parts(x);
    u[i] = pack2(f.x, f.y);
  }
  __device__ __forceinline__ void put_element(int i, bf16 x) {
    const uint32_t b = __bfloat16_as_ushort(x);
    u[i >> 1] = (i & 1) ? (u[i >> 1] & 0xffffu) | (b << 16) : (u[i >> 1] & 0xffff0000u) | b;
  }
  __device__ __forceinline__ bf16 element(int i) const {
    return __ushort_as_bfloat16((unsigned short)((i & 1) ? u[i >> 1] >> 16 : u[i >> 1] & 0xffffu));
  }
  __device__ __forceinline__ void clear() { u[0] = u[1] = u[2] = u[3] = 0; }
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+r"(u[i]));
  }
};

template <>
struct Raw<bf16, 1> {
  bf16 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *p; }
  __device__ __forceinline__ void store(bf16* p) const { *p = v; }
  __device__ __forceinline__ float get(int) const { return __bfloat162float(v); }
  __device__ __forceinline__ void set(const float* f) { v = __float2bfloat16_rn(f[0]); }
  __device__ __forceinline__ float unit(int) const { return __bfloat162float(v); }
  __device__ __forceinline__ void put(int, float f) { v = __float2bfloat16_rn(f); }
  __device__ __forceinline__ void put_element(int, bf16 x) { v = x; }
  __device__ __forceinline__ bf16 element(int) const { return v; }
  __device__ __forceinline__ void clear() { v = __ushort_as_bfloat16(0); }
  __device__ __forceinline__ void renew() {}
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
  __device__ __forceinline__ F2 unit(int i) const { return pair(v[2 * i], v[2 * i + 1]); }
  __device__ __forceinline__ void put(int i, F2 x) {
    const float2 f = parts(x);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
  __device__ __forceinline__ void put_element(int i, float x) { v[i] = x; }
  __device__ __forceinline__ float element(int i) const { return v[i]; }
  __device__ __forceinline__ void clear() { v[0] = v[1] = v[2] = v[3] = 0.f; }
  __device__ __forceinline__ void renew() {}
};

template <>
struct Raw<float, 8> {
  Raw<float, 4> a, b;
  __device__ __forceinline__ void load(const float* p) { a.load(p), b.load(p + 4); }
  __device__ __forceinline__ F2 unit(int i) const { return i < 2 ? a.unit(i) : b.unit(i - 2); }
};

template <>
struct Raw<float, 1> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ void store(float* p) const { *p = v; }
  __device__ __forceinline__ float get(int) const { return v; }
  __device__ __forceinline__ void set(const float* f) { v = f[0]; }
  __device__ __forceinline__ float unit(int) const { return v; }
  __device__ __forceinline__ void put(int, float f) { v = f; }
  __device__ __forceinline__ void put_element(int, float x) { v = x; }
  __device__ __forceinline__ float element(int) const { return v; }
  __device__ __forceinline__ void clear() { v = 0.f; }
  __device__ __forceinline__ void renew() {}
};

// Elements of T in 16 bytes.
template <typename T>
constexpr int kFull = 16 / (int)sizeof(T);

}  // namespace row
}  // namespace fbob
