// Layer norm, backward: with a = w o dy,
//   dx = r (a - m(a) - xh m(a xh)),  dw = sum over rows of dy xh,  db = sum of dy.
// One read of x and dy; the column sums are kept in registers over a block's
// rows, written once per block and added up by a second kernel in a fixed
// order, so the result does not depend on timing.
#include <initializer_list>
#include <type_traits>

#include "layer_norm.cuh"

namespace fbob {
namespace ln {
namespace {

template <typename T, typename WT, int VEC, int E, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : kWarps * 32)
    bwd_kernel(const T* x, const WT* w, const float* mean, const float* rstd, const T* dy, T* dx, float* dw_parts,
               float* db_parts, long long rows, int D) {
  extern __shared__ float sh[];
  const Cols<VEC, E, BLOCK> c;
  const long long step = BLOCK ? gridDim.x : (long long)gridDim.x * kWarps;
  const float inv = 1.f / (float)D;
  float dw[E] = {}, db[E] = {};
  for (long long r = BLOCK ? blockIdx.x : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += step) {
    Raw<T, VEC> vx[c.NV], vd[c.NV];
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
        vx[i].load(x + r * D + c.at(i));
        vd[i].load(dy + r * D + c.at(i));
      }
    }
    const float mu = mean[r], rs = rstd[r];
    float s[2] = {0.f, 0.f};  // sums of a, a xh
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
      if (c.at(i) < D) {
        Raw<WT, VEC> q;
        if (w) q.load(w + c.at(i));
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (vx[i].get(j) - mu) * rs, g = vd[i].get(j);
          const float a = w ? g * q.get(j) : g;
          s[0] += a;
          s[1] += a * xh;
          dw[i * VEC + j] += g * xh;
          db[i * VEC + j] += g;
        }
      }
    }
    row_sum<2, BLOCK>(s);
    const float ma = s[0] * inv, max_ = s[1] * inv;
    if (dx) {
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
        if (c.at(i) < D) {
          Raw<WT, VEC> q;
          if (w) q.load(w + c.at(i));
          float o[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float xh = (vx[i].get(j) - mu) * rs, g = vd[i].get(j);
            o[j] = rs * ((w ? g * q.get(j) : g) - ma - xh * max_);
          }
          vd[i].set(o);
          vd[i].store(dx + r * D + c.at(i));
        }
      }
    }
  }
  if (dw_parts) write_column_sums<VEC, E, BLOCK>(dw, dw_parts + (size_t)blockIdx.x * D, D, sh);
  if (db_parts) write_column_sums<VEC, E, BLOCK>(db, db_parts + (size_t)blockIdx.x * D, D, sh);
}

constexpr int kRedCols = 32, kRedRows = 32;

__global__ void __launch_bounds__(kRedCols * kRedRows)
    reduce_kernel(const float* in, int parts, int D, void* out0, void* out1, int out_bf16) {
  __shared__ float sh[kRedRows][kRedCols + 1];
  void* out = blockIdx.y == 0 ? out0 : out1;
  const int col = blockIdx.x * kRedCols + threadIdx.x;
  float t = 0.f;
  if (col < D) {
    const float* src = in + (size_t)blockIdx.y * parts * D + col;
    for (int r = threadIdx.y; r < parts; r += kRedRows) t += src[(size_t)r * D];
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
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const bool vec = a.D % row::kFull<T> == 0 && all_aligned({a.x, a.w, a.dy, a.dx});
  const Shape sh = shape(a.rows, a.D, kMaxParts);
  // dw's partial sums first where both are wanted
  float* dwp = a.dw ? a.ws : nullptr;
  float* dbp = a.db ? a.ws + (a.dw ? (size_t)sh.blocks * a.D : 0) : nullptr;
  const int smem = sh.block ? 0 : kWarps * kWarpCols * (int)sizeof(float);
  prof_begin(s, "layer_norm_bwd");
  dispatch<T>(a.D, vec, [&](auto v, auto e, auto block) {
    bwd_kernel<T, WT, v(), e(), block()><<<sh.blocks, sh.threads, smem, s>>>(
        static_cast<const T*>(a.x), static_cast<const WT*>(a.w), a.mean, a.rstd, static_cast<const T*>(a.dy),
        static_cast<T*>(a.dx), dwp, dbp, a.rows, a.D);
  });
  prof_end(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  return reduce_parts(a.ws, sh.blocks, a.D, a.dw ? a.dw : a.db, a.dw ? a.db : nullptr, a.wbf16, s);
}

}  // namespace

cudaError_t reduce_parts(const float* in, int parts, int D, void* out0, void* out1, bool out_bf16, cudaStream_t s) {
  prof_begin(s, "layer_norm_columns");
  reduce_kernel<<<dim3((D + kRedCols - 1) / kRedCols, out1 ? 2 : 1), dim3(kRedCols, kRedRows), 0, s>>>(
      in, parts, D, out0, out1, out_bf16);
  prof_end(s);
  return cudaGetLastError();
}

}  // namespace ln

size_t layer_norm_workspace_floats(long long rows, int D) {
  return 2 * (size_t)ln::shape(rows, D, ln::kMaxParts).blocks * D;
}

cudaError_t layer_norm_bwd(const NormArgs& a, cudaStream_t s) {
  if (!a.bf16) return ln::launch<float, float>(a, s);
  return a.wbf16 ? ln::launch<row::bf16, row::bf16>(a, s) : ln::launch<row::bf16, float>(a, s);
}

}  // namespace fbob
