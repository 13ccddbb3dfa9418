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
// The differences cancel where u and a have a common level L times their spread;
// so does P u, and forming it first and then its product's mean, for one more
// reduction, is as badly off: errors of gx relative to its size, D = 768, level 1
// / 10 / 100: 1.4e-6 / 1.3e-4 / 1.4e-2 here, 1.0e-6 / 0.8e-4 / 0.9e-2 that way.
// One read of x, dy and u; one write of gx and gdy.
#include <initializer_list>
#include <type_traits>

#include "launch.cuh"
#include "layer_norm.cuh"

namespace fbob {
namespace ln {
namespace {

template <typename T, typename WT, int VEC, int E, int OWN, bool EVEN>
__global__ void __launch_bounds__(kMaxThreads<OWN>, kResident<T, E, OWN>)
    bob_kernel(const T* x, const WT* w, const float* mean, const float* rstd, const T* dy, const T* u, const WT* uw,
               const WT* ub, T* gx, T* gdy, float* gw_parts, long long rows, int D, int period, int stages,
               unsigned int* err, unsigned long long wait_ns) {
  constexpr int R = kRows<T, E, 3>, U = kUnits<VEC>;
  using G = Ring<T, 3, R, VEC, OWN, EVEN>;
  extern __shared__ __align__(16) char dyn[];
  allow_next();
  wait_previous();
  __shared__ typename G::Bars bars;
  const T* const tensors[] = {x, dy, u};
  char* const slots =
      dyn + (kStaged<VEC, EVEN> ? ((w != nullptr) + (uw != nullptr) + (ub != nullptr)) * Weights<WT, VEC, E, OWN, EVEN>::bytes(D) : 0);
  const G ring(tensors, rows, D, period, stages, slots, bars);
  const Cols<VEC, E, OWN, EVEN> c(D, VEC == 1 ? 0 : ring.shift());
  char* free = dyn;
  const Weights<WT, VEC, E, OWN, EVEN> ww(w, free, c), wu(uw, free, c), wb(ub, free, c);
  __syncthreads();
  const float inv = 1.f / (float)D;
  int flip = 0;
  Unit<VEC> gw[1][c.NV][U];
#pragma unroll
  for (int i = 0; i < c.NV; ++i) {
#pragma unroll
    for (int e = 0; e < U; ++e) gw[0][i][e] = all<VEC>(0.f);
  }
  float mu_next[R], rs_next[R];  // the rows' statistics, read one step ahead
  auto statistics = [&](long long first) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const long long at = first + j * ring.period;
      mu_next[j] = at < rows ? mean[at] : 0.f;
      rs_next[j] = at < rows ? rstd[at] : 0.f;
    }
  };
  long long r = ring.first;
  statistics(r);
  for (int k = 0; r < rows; ++k, r += ring.step) {
    float mu[R], rs[R];
#pragma unroll
    for (int j = 0; j < R; ++j) mu[j] = mu_next[j], rs[j] = rs_next[j];
    statistics(r + ring.step);
    Raw<T, VEC> vx[R][c.NV], vd[R][c.NV], vu[R][c.NV];
    if (!ring.wait(k, r, err, wait_ns)) return;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      ring.template read<E>(k, r, j, 0, vx[j], c);
      ring.template read<E>(k, r, j, 1, vd[j], c);
      ring.template read<E>(k, r, j, 2, vu[j], c);
    }
    if (OWN == kWarp) {
      __syncwarp();  // the whole warp has read its slots
      ring.fill(k + stages, r + stages * ring.step);
    }
    // columns outside the row hold dy = u = 0, so every term there is zero
    float s[7 * R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      Unit<VEC> t[7];
#pragma unroll
      for (int q = 0; q < 7; ++q) t[q] = all<VEC>(0.f);
      const Unit<VEC> m = all<VEC>(-mu[j]), ir = all<VEC>(rs[j]);
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
        if (!c.any(i)) continue;
        Unit<VEC> qw[U], qu[U];
        ww.load(i, qw, 1.f, c);
        wu.load(i, qu, 0.f, c);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const Unit<VEC> xh = (vx[j][i].unit(e) + m) * ir, g = vd[j][i].unit(e), uu = vu[j][i].unit(e);
          const Unit<VEC> a = g * qw[e], h = g * qu[e];
          t[0] = t[0] + a;
          t[1] = mad(a, xh, t[1]);
          t[2] = t[2] + uu;
          t[3] = mad(uu, xh, t[3]);
          t[4] = mad(uu, a, t[4]);
          t[5] = t[5] + h;
          t[6] = mad(h, xh, t[6]);
        }
      }
#pragma unroll
      for (int q = 0; q < 7; ++q) s[7 * j + q] = total(t[q]);
    }
    row_sum<7 * R, OWN>(s, flip);
    if (OWN != kWarp) ring.fill(k + stages, r + stages * ring.step);  // the sum's barrier followed every read
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const float* t = s + 7 * j;
      const float ma = t[0] * inv, max_ = t[1] * inv, mu_ = t[2] * inv, mux = t[3] * inv;
      const float mpa = t[4] * inv - mu_ * ma - mux * max_;
      const float mh = t[5] * inv - rs[j] * (ma * mux + mu_ * max_);
      const float mhx = t[6] * inv - 2.f * rs[j] * max_ * mux;
      const Unit<VEC> m = all<VEC>(-mu[j]), ir = all<VEC>(rs[j]);
      const Unit<VEC> n_mu = all<VEC>(-mu_), n_mux = all<VEC>(-mux), n_mh = all<VEC>(-mh);
      const Unit<VEC> r_mux = all<VEC>(-rs[j] * mux), r_max = all<VEC>(-rs[j] * max_);
      const Unit<VEC> n_mhx = all<VEC>(-(mhx + rs[j] * mpa));
      const bool live = ring.live(r, j);
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
        if (!c.any(i)) continue;
        vx[j][i].renew(), vd[j][i].renew(), vu[j][i].renew();
        Unit<VEC> qw[U], qu[U], qb[U];
        ww.load(i, qw, 1.f, c);
        wu.load(i, qu, 0.f, c);
        wb.load(i, qb, 0.f, c);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const Unit<VEC> xh = (vx[j][i].unit(e) + m) * ir, g = vd[j][i].unit(e), uu = vu[j][i].unit(e);
          const Unit<VEC> pu = ir * mad(xh, n_mux, uu + n_mu);  // r P u
          const Unit<VEC> h = mad(uu, r_max, g * mad(qw[e], r_mux, qu[e]));
          gw[0][i][e] = mad(pu, g, gw[0][i][e]);
          vx[j][i].put(e, ir * mad(xh, n_mhx, h + n_mh));
          vd[j][i].put(e, mad(qw[e], pu, mad(qu[e], xh, qb[e])));
        }
        if (gx && live) write<T, VEC, E, OWN, EVEN>(gx + (r + j * ring.period) * D, vx[j][i], i, c);
        if (gdy && live) write<T, VEC, E, OWN, EVEN>(gdy + (r + j * ring.period) * D, vd[j][i], i, c);
      }
    }
  }
  float* const parts[] = {gw_parts ? gw_parts + (size_t)blockIdx.x * D : nullptr};
  write_column_sums<1, VEC, E, OWN, EVEN>(gw, parts, reinterpret_cast<float*>(slots), c);  // every copy has been read
}

template <typename T, typename WT>
cudaError_t launch(const NormArgs& a, const DevCtx& ctx, cudaStream_t s) {
  const Layout l = layout<T>(a.D, {a.x, a.dy, a.ux, a.gx, a.gdy}, {a.w, a.uw, a.ub});
  const Shape sh = shape(a.rows, l, kMaxParts);
  cudaError_t e_ = cudaSuccess;
  prof_begin(s, "layer_norm_bob");
  dispatch<T>(l, [&](auto v, auto e, auto own, auto even) {
    auto kernel = bob_kernel<T, WT, v(), e(), own(), even()>;
    int smem = 0;
    const int stages = ring_stages<T, WT, 3, v(), e(), own(), even()>(a.D, a.rows, l, sh, !!a.w + !!a.uw + !!a.ub, a.gw ? 1 : 0, &smem);
    e_ = launch_rows(kernel, sh, smem, s, static_cast<const T*>(a.x), static_cast<const WT*>(a.w), a.mean, a.rstd, static_cast<const T*>(a.dy), static_cast<const T*>(a.ux), static_cast<const WT*>(a.uw), static_cast<const WT*>(a.ub), static_cast<T*>(a.gx), static_cast<T*>(a.gdy), a.gw ? a.ws : nullptr, a.rows, a.D, l.period, stages, ctx.err, ctx.wait_ns);
  });
  prof_end(s);
  const cudaError_t e = e_ != cudaSuccess ? e_ : cudaGetLastError();
  if (e != cudaSuccess || !a.gw) return e;
  return reduce_parts(a.ws, sh.blocks, a.D, a.gw, nullptr, a.wbf16, s);
}

}  // namespace
}  // namespace ln

cudaError_t layer_norm_bob(const NormArgs& a, const DevCtx& c, cudaStream_t s) {
  if (!a.bf16) return ln::launch<float, float>(a, c, s);
  return a.wbf16 ? ln::launch<row::bf16, row::bf16>(a, c, s) : ln::launch<row::bf16, float>(a, c, s);
}

}  // namespace fbob
