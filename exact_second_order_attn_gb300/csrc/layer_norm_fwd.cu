// Layer norm, forward: one read of x, one write of y, and the row statistics
// (mean, r) in fp32 for the backward passes.
#include <initializer_list>
#include <type_traits>

#include "launch.cuh"
#include "layer_norm.cuh"

namespace fbob {
namespace ln {
namespace {

template <typename T, typename WT, int VEC, int E, int OWN, bool EVEN>
__global__ void __launch_bounds__(kMaxThreads<OWN>, kResident<T, E, OWN>)
    fwd_kernel(const T* x, const WT* w, const WT* b, T* y, float* mean, float* rstd, long long rows, int D, float eps,
               int period, int stages, unsigned int* err, unsigned long long wait_ns) {
  constexpr int R = kRows<T, E, 1>, U = kUnits<VEC>;
  using G = Ring<T, 1, R, VEC, OWN, EVEN>;
  extern __shared__ __align__(16) char dyn[];
  allow_next();
  wait_previous();
  __shared__ typename G::Bars bars;
  const T* const tensors[] = {x};
  const int fixed = kStaged<VEC, EVEN> ? ((w != nullptr) + (b != nullptr)) * Weights<WT, VEC, E, OWN, EVEN>::bytes(D) : 0;
  const G ring(tensors, rows, D, period, stages, dyn + fixed, bars);
  const Cols<VEC, E, OWN, EVEN> c(D, VEC == 1 ? 0 : ring.shift());
  char* free = dyn;
  const Weights<WT, VEC, E, OWN, EVEN> ww(w, free, c), wb(b, free, c);
  __syncthreads();
  const float inv = 1.f / (float)D;
  int flip = 0;
  long long r = ring.first;
  for (int k = 0; r < rows; ++k, r += ring.step) {
    Raw<T, VEC> v[R][c.NV];
    if (!ring.wait(k, r, err, wait_ns)) return;
#pragma unroll
    for (int j = 0; j < R; ++j) ring.template read<E>(k, r, j, 0, v[j], c);
    if (OWN == kWarp) {
      __syncwarp();  // the whole warp has read its slots
      ring.fill(k + stages, r + stages * ring.step);
    }
    float s[R], mu[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      Unit<VEC> t = all<VEC>(0.f);
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
#pragma unroll
        for (int e = 0; e < U; ++e) t = t + v[j][i].unit(e);
      }
      s[j] = total(t);
    }
    row_sum<R, OWN>(s, flip);
    if (OWN != kWarp) ring.fill(k + stages, r + stages * ring.step);  // the sum's barrier followed every read
#pragma unroll
    for (int j = 0; j < R; ++j) {
      mu[j] = s[j] * inv;
      Unit<VEC> t = all<VEC>(0.f);
      const Unit<VEC> m = all<VEC>(-mu[j]);
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
        if (!c.any(i)) continue;
        if (c.whole(i)) {
#pragma unroll
          for (int e = 0; e < U; ++e) {
            const Unit<VEC> d = v[j][i].unit(e) + m;
            t = mad(d, d, t);
          }
        } else {
          float f = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float d = (float)v[j][i].element(e) - mu[j];
            f += c.has(i, e) ? d * d : 0.f;
          }
          if constexpr (VEC > 1) t = t + row::pair(f, 0.f);
        }
      }
      s[j] = total(t);
    }
    row_sum<R, OWN>(s, flip);
    float rs[R];
#pragma unroll
    for (int j = 0; j < R; ++j) rs[j] = rsqrtf(s[j] * inv + eps);
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (!c.any(i)) continue;
      Unit<VEC> qw[U], qb[U];
      ww.load(i, qw, 1.f, c);
      wb.load(i, qb, 0.f, c);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const Unit<VEC> m = all<VEC>(-mu[j]), ir = all<VEC>(rs[j]);
#pragma unroll
        for (int e = 0; e < U; ++e) v[j][i].put(e, mad((v[j][i].unit(e) + m) * ir, qw[e], qb[e]));
        if (ring.live(r, j)) write<T, VEC, E, OWN, EVEN>(y + (r + j * ring.period) * D, v[j][i], i, c);
      }
    }
    if (c.lane == 0) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (ring.live(r, j)) {
          mean[(r + j * ring.period)] = mu[j];
          rstd[(r + j * ring.period)] = rs[j];
        }
      }
    }
  }
}

template <typename T, typename WT>
cudaError_t launch(const NormArgs& a, const DevCtx& ctx, cudaStream_t s) {
  const Layout l = layout<T>(a.D, {a.x, a.y}, {a.w, a.b});
  const Shape sh = shape(a.rows, l, 2 * sm_count());
  cudaError_t e_ = cudaSuccess;
  prof_begin(s, "layer_norm_fwd");
  dispatch<T>(l, [&](auto v, auto e, auto own, auto even) {
    auto kernel = fwd_kernel<T, WT, v(), e(), own(), even()>;
    int smem = 0;
    const int stages = ring_stages<T, WT, 1, v(), e(), own(), even()>(a.D, a.rows, l, sh, !!a.w + !!a.b, false, &smem);
    e_ = launch_rows(kernel, sh, smem, s, static_cast<const T*>(a.x), static_cast<const WT*>(a.w), static_cast<const WT*>(a.b), static_cast<T*>(a.y), a.mean, a.rstd, a.rows, a.D, a.eps, l.period, stages, ctx.err, ctx.wait_ns);
  });
  prof_end(s);
  return e_ != cudaSuccess ? e_ : cudaGetLastError();
}

}  // namespace
}  // namespace ln

cudaError_t layer_norm_fwd(const NormArgs& a, const DevCtx& c, cudaStream_t s) {
  if (!a.bf16) return ln::launch<float, float>(a, c, s);
  return a.wbf16 ? ln::launch<row::bf16, row::bf16>(a, c, s) : ln::launch<row::bf16, float>(a, c, s);
}

}  // namespace fbob
