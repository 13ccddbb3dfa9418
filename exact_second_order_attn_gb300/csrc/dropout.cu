// Dropout of a contiguous tensor, added to a residual: y = r + m x (the mask's
// definition is in dropout.cuh).  The map is linear and its own transpose, so
// gradients of any order are the same call.
//
// A thread takes eight columns of a row, the span of one generator call, with
// 16-byte accesses where a row's groups start on 16 bytes.  A block walks over its
// groups with a stride, kGroups of them in flight per thread.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dropout.cuh"
#include "launch.cuh"
#include "prof.h"
#include "vec8.cuh"

namespace fbob {
namespace {

constexpr int kThreads = 256, kGroups = 2;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutArgs a) {
  allow_next();
  wait_previous();
  const Dropper drop(a.drop);
  const unsigned per = (a.D + 7) / 8;
  const long long total = a.rows * per, step = (long long)gridDim.x * kThreads;
  const T *x = static_cast<const T*>(a.x), *r = static_cast<const T*>(a.r);
  T* y = static_cast<T*>(a.y);
  for (long long i0 = (long long)blockIdx.x * kThreads + threadIdx.x; i0 < total; i0 += step * kGroups) {
    float v[kGroups][8], w[kGroups][8];
    unsigned row[kGroups], group[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const long long i = i0 + u * step;
      if (i >= total) break;
      const long long q = total <= 0xffffffffll ? (unsigned)i / per : i / per;
      row[u] = (unsigned)q, group[u] = (unsigned)(i - q * per);
      const long long at = q * a.D + 8ll * group[u];
      load8<T, VEC>(x + at, a.D - 8 * (int)group[u], v[u]);
      if (r) load8<T, VEC>(r + at, a.D - 8 * (int)group[u], w[u]);
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      if (i0 + u * step >= total) break;
      if (drop.on) drop.apply8(group[u], row[u], v[u]);
      if (r) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[u][j] += w[u][j];
      }
      store8<T, VEC>(y + (long long)row[u] * a.D + 8ll * group[u], a.D - 8 * (int)group[u], v[u]);
    }
  }
}

template <typename T, bool VEC>
cudaError_t launch(const DropoutArgs& a, cudaStream_t s) {
  const long long total = a.rows * ((a.D + 7) / 8), each = (long long)kThreads * kGroups;
  const long long blocks = (total + each - 1) / each, most = 8ll * sm_count();
  prof_begin(s, "dropout");
  const cudaError_t e =
      chained(dropout_kernel<T, VEC>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, 1, s, a);
  prof_end(s);
  return e;
}

}  // namespace

cudaError_t dropout(const DropoutArgs& a, cudaStream_t s) {
  const uintptr_t all = (uintptr_t)a.x | (uintptr_t)a.r | (uintptr_t)a.y;
  const bool vec = a.D % 8 == 0 && all % 16 == 0;
  if (a.bf16) return vec ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
  return vec ? launch<float, true>(a, s) : launch<float, false>(a, s);
}

}  // namespace fbob
