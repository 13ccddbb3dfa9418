// Layer norm over rows of D elements: what its three kernels share.
//
//   y = w xh + b,  xh = (x - m(x)) r,  r = (m((x - m(x))^2) + eps)^(-1/2)
//
// with m() the mean over the row.  The kernels are bound by memory, so a row
// is read once and kept in registers between its reductions, in its memory
// format.  A row belongs to a warp up to 1024 columns and to a whole thread
// block of ceil(D / 16) threads above that, so that each thread holds at most
// 32 (16) elements of it.  Row statistics are fp32 and two-pass: the variance
// is summed over x - m(x), not over x^2.
#pragma once

#include <cuda_runtime.h>

#include "internal.h"
#include "prof.h"
#include "rowvec.cuh"

namespace fbob {
namespace ln {

using row::bf16;
using row::Raw;

constexpr int kWarps = 8;         // rows in flight per block when a warp owns a row
constexpr int kWarpCols = 1024;   // widest row of one warp
constexpr int kBlockElems = 16;   // elements per thread when a block owns a row

// The columns of a thread: vector i (of VEC) starts at (i * threads + lane) * VEC.
template <int VEC, int E, bool BLOCK>
struct Cols {
  static constexpr int NV = E / VEC;
  int lane, threads;
  __device__ __forceinline__ Cols()
      : lane(BLOCK ? threadIdx.x : threadIdx.x & 31), threads(BLOCK ? blockDim.x : 32) {}
  __device__ __forceinline__ int at(int i) const { return (i * threads + lane) * VEC; }
};

// Sums of K values over the threads of a row; every thread gets them.
template <int K, bool BLOCK>
__device__ __forceinline__ void row_sum(float (&v)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if constexpr (BLOCK) {
    __shared__ float part[K][32];
    const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    __syncthreads();  // the previous use of `part` has been read
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) part[k][w] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = 0.f;
      for (int i = 0; i < nw; ++i) t += part[k][i];
      v[k] = t;
    }
  }
}

// Each block adds up its rows' contributions to a column sum in registers
// (acc); this writes the block's own total to out[D], summed over its warps in
// a fixed order.  sh: kWarps x kWarpCols floats (unused when BLOCK).
template <int VEC, int E, bool BLOCK>
__device__ __forceinline__ void write_column_sums(const float (&acc)[E], float* out, int D, float* sh) {
  const Cols<VEC, E, BLOCK> c;
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[c.at(i) + j] = acc[i * VEC + j];
      }
    }
  } else {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) sh[(threadIdx.x >> 5) * kWarpCols + c.at(i) + j] = acc[i * VEC + j];
      }
    }
    __syncthreads();
    for (int col = threadIdx.x; col < D; col += blockDim.x) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += sh[w * kWarpCols + col];
      out[col] = t;
    }
  }
}

// Launch shape: `rows` rows of D columns, at most max_blocks blocks that walk
// over the rows.
struct Shape {
  bool block;
  int threads, blocks;
};
inline Shape shape(long long rows, int D, int max_blocks) {
  Shape s;
  s.block = D > kWarpCols;
  s.threads = s.block ? ((D + kBlockElems - 1) / kBlockElems + 31) / 32 * 32 : kWarps * 32;
  const long long want = s.block ? rows : (rows + kWarps - 1) / kWarps;
  s.blocks = (int)(want < max_blocks ? want : max_blocks);
  return s;
}

// Calls f with the compile-time (VEC, E, BLOCK) of a launch.
template <typename T, typename F>
inline void dispatch(int D, bool vec, F&& f) {
  constexpr int V = row::kFull<T>;
  auto with = [&](auto e, auto block) {
    if (vec) f(std::integral_constant<int, V>{}, e, block);
    else f(std::integral_constant<int, 1>{}, e, block);
  };
  if (D > kWarpCols) with(std::integral_constant<int, kBlockElems>{}, std::true_type{});
  else if (D <= 256) with(std::integral_constant<int, 8>{}, std::false_type{});
  else if (D <= 512) with(std::integral_constant<int, 16>{}, std::false_type{});
  else if (D <= 768) with(std::integral_constant<int, 24>{}, std::false_type{});
  else with(std::integral_constant<int, 32>{}, std::false_type{});
}

inline bool all_aligned(std::initializer_list<const void*> ps) {
  uintptr_t bits = 0;
  for (const void* p : ps) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & 15u) == 0;
}

// Blocks of the kernels that reduce over rows (one partial sum row each).  A
// constant, so that the workspace depends on the sizes alone.
constexpr int kMaxParts = 608;

// Adds up `parts` partial rows in[k][parts][D] into out_k[D] (k < n).
cudaError_t reduce_parts(const float* in, int parts, int D, void* out0, void* out1, bool out_bf16, cudaStream_t s);

}  // namespace ln
}  // namespace fbob
