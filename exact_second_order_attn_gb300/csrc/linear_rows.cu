// A linear layer of few tokens: one token is bound by reading W (4096 -> 16,384, bf16,
// 23.6 us: 5.7 TB/s), more by the issue of their products, some 7 per picosecond, where a
// tensor-core tile of 256 rows takes the same time for 16 as for one.  takes_rows() is where
// the two meet.  us of a call, here / in tiles:
//                            1 token      2           4           8           16
//   bf16   768 ->  2304     2.6 /  7.0   3.0 /  6.9  3.5 /  6.9  4.3 /  7.4   6.4 /  7.4
//         2048 ->  2048     3.5 /  8.1   5.5 /  8.1  6.1 /  8.2  8.3 /  8.1  12.1 /  8.3
//         4096 ->  4096     7.5 / 14.0  13.2 / 13.7 16.2 / 13.2 23.3 / 13.8  37.8 / 12.0
//         4096 -> 16,384   23.6 / 35.9  45.7 / 34.1 61.8 / 38.0 92.3 / 33.2 163   / 28.5
//         4097 ->  4096    13.3 / 26.9  16.7 / 26.8 22.0 / 27.0 29.1 / 26.4  46.2 / 23.3
//   fp32   768 ->  2304     3.3 / 16.8   3.5 / 16.8  3.9 / 16.2  4.7 / 16.1   6.7 / 16.0
//         4096 ->  4096    14.2 / 63.0  15.9 / 64.1 19.8 / 65.7 25.6 / 65.9  40.2 / 66.2
//         4096 -> 16,384   47.8 / 218   54.9 / 218  86.3 / 218  143  / 219   263  / 220
//
// A warp takes four rows of W (outputs) and all tokens; a lane eight columns per step,
// so every 16 bytes of W serve all tokens and x comes from the L1 cache.  Sums are
// fp32.  Where the outputs alone do not fill the device, 2, 4 or 8 warps of a block
// share the contraction of the same outputs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "dropout.cuh"
#include "launch.cuh"
#include "linear.h"
#include "prof.h"
#include "vec8.cuh"

namespace fbob {
namespace lin {
namespace {

constexpr int kWarps = 8, kOutputs = 4;  // warps of a block, outputs of a warp

// Sums of NV (a power of two up to 32) values over the lanes: lane l returns that of
// value l >> (5 - log2 NV).
template <int NV>
__device__ __forceinline__ float sum_lanes(float* v) {
  const int lane = threadIdx.x & 31;
  int n = NV;
#pragma unroll
  for (int h = 16; h > 0; h >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & h;
#pragma unroll
      for (int j = 0; j < NV / 2; ++j) {
        if (j < n) {
          const float give = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
          v[j] = keep + __shfl_xor_sync(0xffffffffu, give, h);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], h);
    }
  }
  return v[0];
}

// Eight columns of a row for this lane: neighbours (VEC), or every 32nd one, which
// needs no alignment.
template <typename E, bool VEC>
__device__ __forceinline__ void lane8(const E* row, int k0, int K, float* v) {
  if constexpr (VEC) {
    load8<E, true>(row + k0 + 8 * (threadIdx.x & 31), 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = k0 + 32 * j + (int)(threadIdx.x & 31);
      v[j] = k < K ? (float)row[k] : 0.f;
    }
  }
}

template <typename E, int TT, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, TT >= 8 ? 2 : 3)
    rows_kernel(const E* x, const E* W, const E* bias, const E* r, E* y, Kept<E>* z, int T, int K, int N, int act, const __grid_constant__ DropArgs da,
                int share) {
  allow_next();
  wait_previous();
  constexpr int NV = kOutputs * TT, SETS = NV > 32 ? NV / 32 : 1, PER = NV / SETS;
  __shared__ float part[kWarps][NV];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / share, turn = warp % share;
  const int n0 = (int)(blockIdx.x * (kWarps / share) + group) * kOutputs;
  float sum[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) sum[j] = 0.f;
  if (n0 < N) {
#pragma unroll(TT > 4 ? 1 : 2)
    for (int k0 = turn * 256; k0 < K; k0 += share * 256) {
      const bool in = !VEC || k0 + 8 * lane < K;  // K is a multiple of 8 where VEC
      if (in) {
        float w[kOutputs][8];
#pragma unroll
        for (int o = 0; o < kOutputs; ++o)
          lane8<E, VEC>(W + (size_t)(n0 + o < N ? n0 + o : N - 1) * K, k0, K, w[o]);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          if (t < T) {
            float v[8];
            lane8<E, VEC>(x + (size_t)t * K, k0, K, v);
#pragma unroll
            for (int o = 0; o < kOutputs; ++o) {
#pragma unroll
              for (int j = 0; j < 8; ++j) sum[o * TT + t] = fmaf(w[o][j], v[j], sum[o * TT + t]);
            }
          }
        }
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const float s = sum_lanes<PER>(sum + i * PER);
    constexpr int each = 32 / PER;
    if (lane % each == 0) part[warp][i * PER + lane / each] = s;
  }
  __syncthreads();
  if (n0 >= N) return;
  const Dropper drop(da);
  for (int j = turn * 32 + lane; j < NV; j += share * 32) {
    const int n = n0 + j / TT, t = j % TT;
    if (n >= N || t >= T) continue;
    float v = 0.f;
    for (int w = 0; w < share; ++w) v += part[group * share + w][j];
    const size_t at = (size_t)t * N + n;
    if (bias) v += (float)bias[n];
    if (z) {
      const float kept = sizeof(E) == 2 && act == kActRelu ? kept_sign(v) : v;
      store8<Kept<E>, false>(z + at, 1, &kept);
    }
    v = act_value<sizeof(E) == 4>(act, v);
    if (drop.on) {
      float m[8];
      drop.factors8((uint32_t)(n >> 3), (uint32_t)t, m);
      float f = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) f = (n & 7) == q ? m[q] : f;
      v = f != 0.f ? v * f : 0.f;
    }
    if (r) v += (float)r[at];
    y[at] = (E)v;
  }
}

template <typename E, int TT, bool VEC>
cudaError_t launch_as(const LinearArgs& a, cudaStream_t s) {
  // warps that share a contraction: until two blocks a multiprocessor are there, or a
  // warp has a single step
  const long long groups = ((long long)a.N + kOutputs - 1) / kOutputs;
  int share = 1;
  while (share < kWarps && groups * share < 2ll * 152 * kWarps && share * 256 < a.K) share *= 2;
  const int per = kWarps / share;
  prof_begin(s, "linear_rows");
  const cudaError_t e = chained(
      rows_kernel<E, TT, VEC>, dim3((unsigned)((groups + per - 1) / per)), dim3(kWarps * 32), 0, 1, s,
      static_cast<const E*>(a.x), static_cast<const E*>(a.W), static_cast<const E*>(a.b), static_cast<const E*>(a.r),
      static_cast<E*>(a.y), static_cast<Kept<E>*>(a.z_out), a.T, a.K, a.N, a.act, a.drop, share);
  prof_end(s);
  return e;
}

template <typename E, bool VEC>
cudaError_t launch(const LinearArgs& a, cudaStream_t s) {
  if (a.T <= 1) return launch_as<E, 1, VEC>(a, s);
  if (a.T <= 2) return launch_as<E, 2, VEC>(a, s);
  if (a.T <= 4) return launch_as<E, 4, VEC>(a, s);
  if (a.T <= 8) return launch_as<E, 8, VEC>(a, s);
  return launch_as<E, 16, VEC>(a, s);
}

}  // namespace

cudaError_t rows(const LinearArgs& a, cudaStream_t s) {
  const bool vec = a.K % 8 == 0 && ((uintptr_t)a.x | (uintptr_t)a.W) % 16 == 0;
  if (a.bf16) return vec ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
  return vec ? launch<float, true>(a, s) : launch<float, false>(a, s);
}

}  // namespace lin
}  // namespace fbob
