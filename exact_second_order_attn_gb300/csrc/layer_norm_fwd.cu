// Layer norm, forward: one read of x, one write of y, and the row statistics
// (mean, r) in fp32 for the backward passes.
#include <initializer_list>
#include <type_traits>

#include "layer_norm.cuh"

namespace fbob {
namespace ln {
namespace {

template <typename T, typename WT, int VEC, int E, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : kWarps * 32)
    fwd_kernel(const T* x, const WT* w, const WT* b, T* y, float* mean, float* rstd, long long rows, int D, float eps) {
  const Cols<VEC, E, BLOCK> c;
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kWarps;
  const float inv = 1.f / (float)D;
  for (long long r = BLOCK ? blockIdx.x : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += step) {
    Raw<T, VEC> v[c.NV];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) v[i].load(x + r * D + c.at(i));
    }
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[0] += v[i].get(j);
      }
    }
    row_sum<1, BLOCK>(s);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float t = v[i].get(j) - mu;
          s[0] += t * t;
        }
      }
    }
    row_sum<1, BLOCK>(s);
    const float rs = rsqrtf(s[0] * inv + eps);
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = (v[i].get(j) - mu) * rs;
        if (w) {
          Raw<WT, VEC> q;
          q.load(w + c.at(i));
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] *= q.get(j);
        }
        if (b) {
          Raw<WT, VEC> q;
          q.load(b + c.at(i));
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] += q.get(j);
        }
        v[i].set(o);
        v[i].store(y + r * D + c.at(i));
      }
    }
    if (c.lane == 0) {
      mean[r] = mu;
      rstd[r] = rs;
    }
  }
}

template <typename T, typename WT>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const bool vec = a.D % row::kFull<T> == 0 && all_aligned({a.x, a.w, a.b, a.y});
  const Shape sh = shape(a.rows, a.D, 16 * sm_count());
  prof_begin(s, "layer_norm_fwd");
  dispatch<T>(a.D, vec, [&](auto v, auto e, auto block) {
    fwd_kernel<T, WT, v(), e(), block()><<<sh.blocks, sh.threads, 0, s>>>(
        static_cast<const T*>(a.x), static_cast<const WT*>(a.w), static_cast<const WT*>(a.b), static_cast<T*>(a.y),
        a.mean, a.rstd, a.rows, a.D, a.eps);
  });
  prof_end(s);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ln

cudaError_t layer_norm_fwd(const NormArgs& a, cudaStream_t s) {
  if (!a.bf16) return ln::launch<float, float>(a, s);
  return a.wbf16 ? ln::launch<row::bf16, row::bf16>(a, s) : ln::launch<row::bf16, float>(a, s);
}

}  // namespace fbob
