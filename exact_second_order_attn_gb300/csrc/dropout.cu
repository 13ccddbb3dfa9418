// Dropout of a contiguous tensor, added to a residual: y = r + m x (the mask's
// definition is in dropout.cuh).  The map is linear and its own transpose, so
// gradients of any order are the same call.
//
// Rows that start on 16 bytes: a thread takes eight columns of a row, the span of one
// generator call, in 16-byte accesses; kGroups of them at once, one of bf16 (32,768 x 4096
// 82 us; four, which leave room for fewer threads, 88), two of fp32 (16,384 x 4096 81 us;
// one 91).
// Other rows: a warp takes 256 columns of a row, an element per lane and step, so that
// accesses stay together; a lane draws for eight of the columns and hands out their
// bits; of rows of up to 128 columns it takes several.  (A thread's eight columns one by
// one: 5003 x 1537 fp32 31 us.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dropout.cuh"
#include "launch.cuh"
#include "prof.h"
#include "vec8.cuh"

namespace fbob {
namespace {

constexpr int kThreads = 256;
template <typename T>
constexpr int kGroups = sizeof(T) == 2 ? 1 : 2;

template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutArgs a) {
  allow_next();
  wait_previous();
  const Dropper drop(a.drop);
  const unsigned per = a.D / 8;
  const long long total = a.rows * per, step = (long long)gridDim.x * kThreads;
  const T *x = static_cast<const T*>(a.x), *r = static_cast<const T*>(a.r);
  T* y = static_cast<T*>(a.y);
  long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  // the place of group i, and how far a step moves it: one division each
  uint32_t row = (uint32_t)(i / per), group = (uint32_t)(i - (long long)row * per);
  const uint32_t rows = (uint32_t)(step / per), groups = (uint32_t)(step - (long long)rows * per);
  while (i < total) {
    Raw8<T> v[kGroups<T>], w[kGroups<T>];
#pragma unroll
    for (int u = 0; u < kGroups<T>; ++u) {
      if (i + u * step < total) {
        v[u].template load<true>(x + 8 * (i + u * step), 8);
        if (r) w[u].template load<true>(r + 8 * (i + u * step), 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kGroups<T>; ++u, i += step) {
      if (i < total) {
        float f[8];
        v[u].values(f);
        if (drop.on) drop.apply8(group, row, f);
        if (r) {
          float g[8];
          w[u].values(g);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] += g[j];
        }
        store8<T, true>(y + 8 * i, 8, f);
      }
      row += rows, group += groups;
      if (group >= per) group -= per, ++row;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_rows_kernel(const __grid_constant__ DropoutArgs a) {
  allow_next();
  wait_previous();
  const Dropper drop(a.drop);
  const int lane = threadIdx.x & 31;
  const unsigned per = (a.D + 255) / 256;
  const long long total = a.rows * per, step = (long long)gridDim.x * (kThreads / 32);
  const T *x = static_cast<const T*>(a.x), *r = static_cast<const T*>(a.r);
  T* y = static_cast<T*>(a.y);
  for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
    const long long row = total <= 0xffffffffll ? (unsigned)i / per : i / per;
    const int c0 = (int)(i - row * per) * 256 + lane;
    const long long at = row * a.D + c0;
    T v[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (c0 + 32 * j < a.D) {
        v[j] = x[at + 32 * j];
        if (r) w[j] = r[at + 32 * j];
      }
    }
    unsigned kept = drop.on ? drop.kept8((uint32_t)(c0 - lane) / 8 + lane, (uint32_t)row) : 0xffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // column 32 j + lane of the 256 is column lane % 8 of the group 4 j + lane / 8
      const unsigned bits = __shfl_sync(0xffffffffu, kept, 4 * j + lane / 8);
      if (c0 + 32 * j < a.D) {
        float f = bits >> (lane & 7) & 1u ? (float)v[j] * drop.scale : 0.f;
        if (r) f += (float)w[j];
        y[at + 32 * j] = (T)f;
      }
    }
  }
}

// Rows of up to 128 columns: a warp takes as many as its lanes' groups hold (`each`),
// which lie one behind the other.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    dropout_short_kernel(const __grid_constant__ DropoutArgs a, int each, unsigned inverse) {
  allow_next();
  wait_previous();
  const Dropper drop(a.drop);
  const int lane = threadIdx.x & 31, groups = (a.D + 7) / 8;
  const long long step = (long long)gridDim.x * (kThreads / 32) * each;
  const T *x = static_cast<const T*>(a.x), *r = static_cast<const T*>(a.r);
  T* y = static_cast<T*>(a.y);
  for (long long r0 = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * each; r0 < a.rows; r0 += step) {
    const int rows = (int)(a.rows - r0 < each ? a.rows - r0 : each), n = rows * a.D;
    const long long at = r0 * a.D + lane;
    T v[8], w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (lane + 32 * j < n) {
        v[j] = x[at + 32 * j];
        if (r) w[j] = r[at + 32 * j];
      }
    }
    const unsigned kept = drop.on ? drop.kept8((uint32_t)(lane % groups), (uint32_t)r0 + lane / groups) : 0xffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane + 32 * j, row = (int)((unsigned)e * inverse >> 16), c = e - row * a.D;
      const unsigned bits = __shfl_sync(0xffffffffu, kept, (row * groups + c / 8) & 31);
      if (e < n) {
        float f = bits >> (c & 7) & 1u ? (float)v[j] * drop.scale : 0.f;
        if (r) f += (float)w[j];
        y[at + 32 * j] = (T)f;
      }
    }
  }
}

template <typename T>
cudaError_t launch(const DropoutArgs& a, bool vec, cudaStream_t s) {
  const int each = a.D <= 128 ? 32 / ((a.D + 7) / 8) : 1;
  const long long units = vec ? a.rows * (a.D / 8) : a.D <= 128 ? (a.rows + each - 1) / each : a.rows * ((a.D + 255) / 256);
  const long long block = vec ? kThreads * kGroups<T> : kThreads / 32;
  const long long blocks = (units + block - 1) / block, most = 16ll * sm_count();
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), threads(kThreads);
  prof_begin(s, "dropout");
  // (the inverse is exact for elements below 256: 65,536 / D rounded up is off by less than 1, 256 times that
  // by less than 65,536 / D)
  const cudaError_t e =
      vec          ? chained(dropout_kernel<T>, grid, threads, 0, 1, s, a)
      : a.D <= 128 ? chained(dropout_short_kernel<T>, grid, threads, 0, 1, s, a, each, 65536u / a.D + 1)
                   : chained(dropout_rows_kernel<T>, grid, threads, 0, 1, s, a);
  prof_end(s);
  return e;
}

}  // namespace

cudaError_t dropout(const DropoutArgs& a, cudaStream_t s) {
  const uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.r | (uintptr_t)a.y;
  const bool vec = a.D % 8 == 0 && all % 16 == 0;
  return a.bf16 ? launch<__nv_bfloat16>(a, vec, s) : launch<float>(a, vec, s);
}

}  // namespace fbob
