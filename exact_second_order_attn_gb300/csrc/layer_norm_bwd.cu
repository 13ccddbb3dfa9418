// Layer norm, backward: with a = w o dy,
//   dx = r (a - m(a) - xh m(a xh)),  dw = sum over rows of dy xh,  db = sum of dy.
// One read of x and dy; the column sums are kept in registers over a block's
// rows, written once per block and added up by a second kernel in a fixed
// order, so the result does not depend on timing.
#include <initializer_list>
#include <type_traits>

#include "launch.cuh"
#include "layer_norm.cuh"

namespace fbob {
namespace ln {
namespace {

template <typename T, typename WT, int VEC, int E, int OWN, bool EVEN>
__global__ void __launch_bounds__(kMaxThreads<OWN>, kResident<T, E, OWN>)
    bwd_kernel(const T* x, const WT* w, const float* mean, const float* rstd, const T* dy, T* dx, float* dw_parts,
               float* db_parts, long long rows, int D, int period, int stages, unsigned int* err,
               unsigned long long wait_ns) {
  constexpr int R = kRows<T, E, 2>, U = kUnits<VEC>;
  using G = Ring<T, 2, R, VEC, OWN, EVEN>;
  extern __shared__ __align__(16) char dyn[];
  allow_next();
  wait_previous();
  __shared__ typename G::Bars bars;
  const T* const tensors[] = {x, dy};
  char* const slots = dyn + (kStaged<VEC, EVEN> && w ? Weights<WT, VEC, E, OWN, EVEN>::bytes(D) : 0);
  const G ring(tensors, rows, D, period, stages, slots, bars);
  const Cols<VEC, E, OWN, EVEN> c(D, VEC == 1 ? 0 : ring.shift());
  char* free = dyn;
  const Weights<WT, VEC, E, OWN, EVEN> ww(w, free, c);
  __syncthreads();
  const float inv = 1.f / (float)D;
  int flip = 0;
  Unit<VEC> sums[2][c.NV][U];  // of dw, db
#pragma unroll
  for (int i = 0; i < c.NV; ++i) {
#pragma unroll
    for (int e = 0; e < U; ++e) sums[0][i][e] = sums[1][i][e] = all<VEC>(0.f);
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
    Raw<T, VEC> vx[R][c.NV], vd[R][c.NV];
    if (!ring.wait(k, r, err, wait_ns)) return;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      ring.template read<E>(k, r, j, 0, vx[j], c);
      ring.template read<E>(k, r, j, 1, vd[j], c);
    }
    if (OWN == kWarp) {
      __syncwarp();  // the whole warp has read its slots
      ring.fill(k + stages, r + stages * ring.step);
    }
    // columns outside the row hold dy = 0, so every term there is zero
    float s[2 * R];  // sums of a, a xh
    Unit<VEC> sa[R], sx[R];
#pragma unroll
    for (int j = 0; j < R; ++j) sa[j] = sx[j] = all<VEC>(0.f);
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (!c.any(i)) continue;
      Unit<VEC> q[U];
      ww.load(i, q, 1.f, c);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const Unit<VEC> m = all<VEC>(-mu[j]), ir = all<VEC>(rs[j]);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const Unit<VEC> xh = (vx[j][i].unit(e) + m) * ir, g = vd[j][i].unit(e), a = g * q[e];
          sa[j] = sa[j] + a;
          sx[j] = mad(a, xh, sx[j]);
          sums[0][i][e] = mad(g, xh, sums[0][i][e]);
          sums[1][i][e] = sums[1][i][e] + g;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) s[2 * j] = total(sa[j]), s[2 * j + 1] = total(sx[j]);
    row_sum<2 * R, OWN>(s, flip);
    if (OWN != kWarp) ring.fill(k + stages, r + stages * ring.step);  // the sum's barrier followed every read
    if (!dx) continue;
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (!c.any(i)) continue;
      Unit<VEC> q[U];
      ww.load(i, q, 1.f, c);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        vx[j][i].renew(), vd[j][i].renew();
        const Unit<VEC> m = all<VEC>(-mu[j]), ir = all<VEC>(rs[j]);
        const Unit<VEC> ma = all<VEC>(-s[2 * j] * inv), max_ = all<VEC>(-s[2 * j + 1] * inv);
#pragma unroll
        for (int e = 0; e < U; ++e) {
          const Unit<VEC> xh = (vx[j][i].unit(e) + m) * ir;
          vd[j][i].put(e, ir * mad(xh, max_, mad(vd[j][i].unit(e), q[e], ma)));
        }
        if (ring.live(r, j)) write<T, VEC, E, OWN, EVEN>(dx + (r + j * ring.period) * D, vd[j][i], i, c);
      }
    }
  }
  float* const parts[] = {dw_parts ? dw_parts + (size_t)blockIdx.x * D : nullptr,
                          db_parts ? db_parts + (size_t)blockIdx.x * D : nullptr};
  write_column_sums<2, VEC, E, OWN, EVEN>(sums, parts, reinterpret_cast<float*>(slots), c);  // every copy has been read
}

constexpr int kRedCols = 32, kRedRows = 32;

__global__ void __launch_bounds__(kRedCols * kRedRows)
    reduce_kernel(const float* in, int parts, int D, void* out0, void* out1, int out_bf16) {
  allow_next();
  wait_previous();
  __shared__ float sh[kRedRows][kRedCols + 1];
  void* out = blockIdx.y == 0 ? out0 : out1;
  const int col = blockIdx.x * kRedCols + threadIdx.x;
  float t = 0.f;
  if (col < D) {
    const float* src = in + (size_t)blockIdx.y * parts * D + col;
    for (int r0 = threadIdx.y; r0 < parts; r0 += 4 * kRedRows) {
      float q[4];  // loads first: their latency would be paid one by one
#pragma unroll
      for (int u = 0; u < 4; ++u) q[u] = r0 + u * kRedRows < parts ? src[(size_t)(r0 + u * kRedRows) * D] : 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u) t += q[u];
    }
  }
  sh[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  // thread (x, y) takes row x of column y, so that a warp adds up one column
  float v = sh[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int c = blockIdx.x * kRedCols + threadIdx.y;
  if (threadIdx.x == 0 && c < D) {
    if (out_bf16) static_cast<bf16*>(out)[c] = __float2bfloat16_rn(v);
    else static_cast<float*>(out)[c] = v;
  }
}

template <typename T, typename WT>
cudaError_t launch(const NormArgs& a, const DevCtx& ctx, cudaStream_t s) {
  const Layout l = layout<T>(a.D, {a.x, a.dy, a.dx}, {a.w});
  const Shape sh = shape(a.rows, l, kMaxParts);
  // dw's partial sums first where both are wanted
  float* dwp = a.dw ? a.ws : nullptr;
  float* dbp = a.db ? a.ws + (a.dw ? (size_t)sh.blocks * a.D : 0) : nullptr;
  cudaError_t e_ = cudaSuccess;
  prof_begin(s, "layer_norm_bwd");
  dispatch<T>(l, [&](auto v, auto e, auto own, auto even) {
    auto kernel = bwd_kernel<T, WT, v(), e(), own(), even()>;
    int smem = 0;
    const int stages = ring_stages<T, WT, 2, v(), e(), own(), even()>(a.D, a.rows, l, sh, !!a.w, a.dw || a.db ? 2 : 0, &smem);
    e_ = launch_rows(kernel, sh, smem, s, static_cast<const T*>(a.x), static_cast<const WT*>(a.w), a.mean, a.rstd, static_cast<const T*>(a.dy), static_cast<T*>(a.dx), dwp, dbp, a.rows, a.D, l.period, stages, ctx.err, ctx.wait_ns);
  });
  prof_end(s);
  const cudaError_t e = e_ != cudaSuccess ? e_ : cudaGetLastError();
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  return reduce_parts(a.ws, sh.blocks, a.D, a.dw ? a.dw : a.db, a.dw ? a.db : nullptr, a.wbf16, s);
}

}  // namespace

cudaError_t reduce_parts(const float* in, int parts, int D, void* out0, void* out1, bool out_bf16, cudaStream_t s) {
  prof_begin(s, "layer_norm_columns");
  const cudaError_t e = chained(reduce_kernel, dim3((D + kRedCols - 1) / kRedCols, out1 ? 2 : 1),
                                dim3(kRedCols, kRedRows), 0, 1, s, in, parts, D, out0, out1, (int)out_bf16);
  prof_end(s);
  return e;
}

}  // namespace ln

size_t layer_norm_workspace_floats(long long rows, int D) {
  // a block per row at most, in whole periods (of up to 8 rows); rows above a
  // warp's but below 2048 columns have up to 128 threads, twice as many blocks
  const long long blocks = (rows + 7) / 8 * 8;
  const int most = (D > ln::kWarpCols - 8 && D <= 2048 ? 2 : 1) * ln::kMaxParts;
  return 2 * (size_t)(blocks < most ? blocks : most) * D;
}

cudaError_t layer_norm_bwd(const NormArgs& a, const DevCtx& c, cudaStream_t s) {
  if (!a.bf16) return ln::launch<float, float>(a, c, s);
  return a.wbf16 ? ln::launch<row::bf16, row::bf16>(a, c, s) : ln::launch<row::bf16, float>(a, c, s);
}

}  // namespace fbob
