// Layer norm, backward over backward: the vector-Jacobian product of
// (x, w, dy) -> (dx, dw, db) along cotangents (u, uw, ub).  With a = w o dy and
// the projection P v = v - m(v) - xh m(v xh) (symmetric), dx = r P a, so
//   f = <u, dx> + <uw, dw> + <ub, db> = sum over rows of r <P u, a> + <uw dy, xh> + <ub, dy>
//   gdy = r w o P u + uw o xh + ub
//   gw  = sum over rows of r P u o dy
// and x enters through xh (whose own product is h -> r P h) and through r
// (dr/dx = -r^2 xh / D):
//   h  = uw o dy - r (a m(u xh) + u m(a xh))
//   gx = r P h - r^2 xh m(P u o a).
// Every mean over the row is one of seven sums taken in one reduction:
//   m(a), m(a xh), m(u), m(u xh), m(u a), m(uw dy), m(uw dy xh), with
//   m(h)    = m(uw dy) - r (m(a) m(u xh) + m(u) m(a xh))
//   m(h xh) = m(uw dy xh) - 2 r m(a xh) m(u xh)
//   m(P u a) = m(u a) - m(u) m(a) - m(u xh) m(a xh).
// One read of x, dy and u; one write of gx and gdy.
#include <initializer_list>
#include <type_traits>

#include "layer_norm.cuh"

namespace fbob {
namespace ln {
namespace {

template <typename T, typename WT, int VEC, int E, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : kWarps * 32)
    bob_kernel(const T* x, const WT* w, const float* mean, const float* rstd, const T* dy, const T* u, const WT* uw,
               const WT* ub, T* gx, T* gdy, float* gw_parts, long long rows, int D) {
  extern __shared__ float sh[];
  const Cols<VEC, E, BLOCK> c;
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kWarps;
  const float inv = 1.f / (float)D;
  float gw[E] = {};
  for (long long r = BLOCK ? blockIdx.x : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += step) {
    Raw<T, VEC> vx[c.NV], vd[c.NV], vu[c.NV];
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
        vx[i].load(x + r * D + c.at(i));
        vd[i].load(dy + r * D + c.at(i));
        vu[i].load(u + r * D + c.at(i));
      }
    }
    const float mu = mean[r], rs = rstd[r];
    float s[7] = {};
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
        Raw<WT, VEC> q, t;
        if (w) q.load(w + c.at(i));
        if (uw) t.load(uw + c.at(i));
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (vx[i].get(j) - mu) * rs, g = vd[i].get(j), uu = vu[i].get(j);
          const float a = w ? g * q.get(j) : g, k = uw ? g * t.get(j) : 0.f;
          s[0] += a;
          s[1] += a * xh;
          s[2] += uu;
          s[3] += uu * xh;
          s[4] += uu * a;
          s[5] += k;
          s[6] += k * xh;
        }
      }
    }
    row_sum<7, BLOCK>(s);
    const float ma = s[0] * inv, max_ = s[1] * inv, mu_ = s[2] * inv, mux = s[3] * inv;
    const float mpa = s[4] * inv - mu_ * ma - mux * max_;
    const float mh = s[5] * inv - rs * (ma * mux + mu_ * max_);
    const float mhx = s[6] * inv - 2.f * rs * max_ * mux;
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
        Raw<WT, VEC> q, t, v;
        if (w) q.load(w + c.at(i));
        if (uw) t.load(uw + c.at(i));
        if (ub) v.load(ub + c.at(i));
        float ox[VEC], od[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (vx[i].get(j) - mu) * rs, g = vd[i].get(j), uu = vu[i].get(j);
          const float wj = w ? q.get(j) : 1.f, tj = uw ? t.get(j) : 0.f;
          const float pu = rs * (uu - mu_ - xh * mux);
          od[j] = wj * pu + tj * xh + (ub ? v.get(j) : 0.f);
          gw[i * VEC + j] += pu * g;
          const float h = tj * g - rs * (wj * g * mux + uu * max_);
          ox[j] = rs * (h - mh - xh * (mhx + rs * mpa));
        }
        vx[i].set(ox);
        vd[i].set(od);
        if (gx) vx[i].store(gx + r * D + c.at(i));
        if (gdy) vd[i].store(gdy + r * D + c.at(i));
      }
    }
  }
  if (gw_parts) write_column_sums<VEC, E, BLOCK>(gw, gw_parts + (size_t)blockIdx.x * D, D, sh);
}

template <typename T, typename WT>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const bool vec =
      a.D % row::kFull<T> == 0 && all_aligned({a.x, a.w, a.dy, a.ux, a.uw, a.ub, a.gx, a.gdy});
  const Shape sh = shape(a.rows, a.D, kMaxParts);
  const int smem = sh.block ? 0 : kWarps * kWarpCols * (int)sizeof(float);
  prof_begin(s, "layer_norm_bob");
  dispatch<T>(a.D, vec, [&](auto v, auto e, auto block) {
    bob_kernel<T, WT, v(), e(), block()><<<sh.blocks, sh.threads, smem, s>>>(
        static_cast<const T*>(a.x), static_cast<const WT*>(a.w), a.mean, a.rstd, static_cast<const T*>(a.dy),
        static_cast<const T*>(a.ux), static_cast<const WT*>(a.uw), static_cast<const WT*>(a.ub),
        static_cast<T*>(a.gx), static_cast<T*>(a.gdy), a.gw ? a.ws : nullptr, a.rows, a.D);
  });
  prof_end(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.gw) return e;
  return reduce_parts(a.ws, sh.blocks, a.D, a.gw, nullptr, a.wbf16, s);
}

}  // namespace
}  // namespace ln

cudaError_t layer_norm_bob(const NormArgs& a, cudaStream_t s) {
  if (!a.bf16) return ln::launch<float, float>(a, s);
  return a.wbf16 ? ln::launch<row::bf16, row::bf16>(a, s) : ln::launch<row::bf16, float>(a, s);
}

}  // namespace fbob
