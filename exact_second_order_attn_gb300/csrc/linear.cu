// Linear layers y = r + m a(x W^T + b): forward, gradients, and the gradients' own
// vector-Jacobian product (formulas in fbob.h; products in linear_gemm.cuh).
//
// Forward: one product whose epilogue adds the bias, applies activation and
// dropout and adds the residual; a training forward also keeps z,
// beside bf16 tensors in fp16: in bf16 its rounding alone made gx and gW 1.53 times
// as far off as a result that is rounded once, where q's and dz's leave 1.41.
// Gradients: dz = m dy a'(z) once (with its column sums, in fp32), then dx = dz W
// and dW = dz^T x; without activation and dropout dz is dy itself.  Second order: one
// product for t whose epilogue turns it into gdy, q and dz, then gx = q W + dz uW and
// gW = q^T x + dz^T ux, each one product over two segments.
//
// dz and q are rounded to bf16 for the products of bf16 tensors, which costs as much
// as the rounding of the result (errors of 1.4 half steps); with up to kExactTokens
// tokens a row of dW hangs on a few of them, and they keep two bf16 terms.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <string.h>

#include "activation.cuh"
#include "ce.h"
#include "dropout.cuh"
#include "launch.cuh"
#include "linear.h"
#include "prof.h"
#include "vec8.cuh"

namespace fbob {
namespace lin {
namespace {

using ce::matrix_map;
using ce::store_map;

size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }
bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

constexpr int kPairs = 76;                     // block pairs of a GB300, for the rule below
constexpr size_t kSlabBytes = 512ull << 20;    // slabs of a product
constexpr long long kLongTerms = 16384;        // bf16 sums above end their chains there

// Times in cycles, estimated, decide between tile widths and numbers of slabs: a step
// of a tile takes 575 (256 columns), 475 or 400 (192, 128: as much of A is loaded for
// fewer products), the hand-over of a tile 1,000; slabs cost a launch and a read of fp32.
double tile_cost(long long steps, int nseg, int tile_n) {
  return (double)steps * nseg * (tile_n == 256 ? 575. : tile_n == 192 ? 475. : 400.) + 1000.;
}
double slab_cost(long long M, long long N, int s) { return s > 1 ? 3500. + 4. * (double)M * (double)N * s / 2500. : 0.; }
long long tiles_of(long long M, long long N, int tile_n) { return ((M + kTileM - 1) / kTileM) * ((N + tile_n - 1) / tile_n); }
bool slabs_fit(long long M, long long N, int s) { return (size_t)M * up(N, 8) * 4 * s <= kSlabBytes; }

// Tile width and slabs of a product of M x N outputs over `steps` steps of the
// contraction in each of nseg segments.
struct Shape {
  int tile_n, splits;
};
Shape choose(long long M, long long N, int steps, int nseg, bool slabs, bool narrow_only) {
  auto cost = [&](int tile, int s) {
    const long long tiles = tiles_of(M, N, tile) * s;
    return (double)((tiles + kPairs - 1) / kPairs) * tile_cost((steps + s - 1) / s, nseg, tile) + slab_cost(M, N, s);
  };
  Shape best{narrow_only ? 128 : 256, 1};
  double least = cost(best.tile_n, 1);
  for (int tile : {192, 128}) {
    if (!narrow_only && cost(tile, 1) < least) best = Shape{tile, 1}, least = cost(tile, 1);
  }
  for (int s = 2; slabs && s <= 64 && s <= steps && slabs_fit(M, N, s); ++s) {
    if (cost(256, s) < least) best = Shape{256, s}, least = cost(256, s);
  }
  return best;
}

// Slabs of two products in one launch (either may be absent: M = 0).  The pairs take
// the tiles of the first, which last longer, then those of the second, in turn.
struct Size {
  long long M, N;
  int steps, nseg;
};
struct Splits {
  int s[2];
};
Splits share(const Size (&z)[2]) {
  Splits best{{1, 1}};
  double least = -1.;
  static constexpr int kTry[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32};  // (the host pays for each pair)
  for (int a : kTry) {
    if (a > 1 && (z[0].M == 0 || a > z[0].steps || !slabs_fit(z[0].M, z[0].N, a))) break;
    for (int b : kTry) {
      if (b > 1 && (z[1].M == 0 || b > z[1].steps || !slabs_fit(z[1].M, z[1].N, b))) break;
      const int s[2] = {a, b};
      long long n[2];
      double each[2], cost = 0.;
      for (int i = 0; i < 2; ++i) {
        n[i] = z[i].M ? tiles_of(z[i].M, z[i].N, 256) * s[i] : 0;
        each[i] = tile_cost((z[i].steps + s[i] - 1) / s[i], z[i].nseg, 256);
        cost += (double)(n[i] / kPairs) * each[i] + (z[i].M ? slab_cost(z[i].M, z[i].N, s[i]) : 0.);
      }
      // what the busiest pair has beyond that: a tile of either, or of both
      const long long r[2] = {n[0] % kPairs, n[1] % kPairs};
      const double most = each[0] > each[1] ? each[0] : each[1];
      cost += r[0] + r[1] > kPairs ? each[0] + each[1] : r[0] && r[1] ? most : r[0] ? each[0] : r[1] ? each[1] : 0.;
      if (least < 0. || cost < least) best = Splits{{a, b}}, least = cost;
    }
  }
  return best;
}

// Where everything lies in the workspace, and the products' shapes.
struct Plan {
  int np, zp;  // bf16 terms of an operand; of dz and q
  int Kp, Np;
  bool copy_k, copy_n;  // [.][K] and [.][N] operands are not read in place
  bool own_dz;          // dz is not dy itself
  bool curved;          // a'' is not zero
  Shape fwd, sec;
  Splits both, dx, dw;  // slabs of dx and dW together, and of each alone
  int sum_rows, sum_parts;
  size_t x, W, ux, uW, dz, q, sums, slab, bytes;
};

int steps_of(long long n) { return (int)((n + kBK - 1) / kBK); }

Plan plan(const LinearArgs& a, LinearPass pass) {
  Plan p;
  const bool bwd = pass == LinearPass::kBwd, bob = pass == LinearPass::kBob;
  p.np = a.bf16 ? 1 : kPlanes;
  p.Kp = (int)up(a.K, 8), p.Np = (int)up(a.N, 8);
  p.copy_k = !a.bf16 || a.K % 8 != 0, p.copy_n = !a.bf16 || a.N % 8 != 0;
  p.own_dz = p.copy_n || a.act != kActNone || a.drop.dropped != 0;
  p.curved = a.act != kActNone && a.act != kActRelu;
  p.zp = !a.bf16 ? kPlanes : p.own_dz && a.T <= kExactTokens ? 2 : 1;
  const int one = a.bf16 ? 1 : 6, back = a.bf16 ? p.zp : 6, two = bob && p.curved ? 2 : 1;
  const bool held = !a.bf16;
  p.fwd = choose(a.T, a.N, steps_of(a.K), one, true, held || a.K > kLongTerms);
  p.sec = choose(a.T, a.N, steps_of(a.K), 2 * one, false, p.zp > 1 || 2ll * a.K > kLongTerms);
  const Size dx{a.T, a.K, steps_of(a.N), back * two}, dw{a.N, a.K, steps_of(a.T), back * two}, none{0, 0, 1, 1};
  if (bwd || bob) p.both = share({dx, dw}), p.dx = share({dx, none}), p.dw = share({none, dw});
  // rows of a block of dz_kernel: as many blocks as fill the device six times
  const long long across = (p.Np + 255) / 256;
  p.sum_rows = (int)up((size_t)((long long)a.T * across / (152 * 6) + 1), 8);
  p.sum_parts = (int)((a.T + p.sum_rows - 1) / p.sum_rows);
  const size_t parts = bob && (a.T + 31) / 32 > p.sum_parts ? (a.T + 31) / 32 : p.sum_parts;
  size_t at = 0;
  auto take = [&](bool want, size_t bytes) {
    const size_t here = at;
    if (want) at += up(bytes, ce::kWorkspaceAlign);
    return here;
  };
  const size_t T = a.T, K = p.Kp, N = p.Np, e = 2 * (size_t)p.np;
  p.x = take(p.copy_k, T * K * e);
  p.W = take(p.copy_k, (size_t)a.N * K * e);
  p.ux = take(bob && p.copy_k, T * K * e);
  p.uW = take(bob && p.copy_k, (size_t)a.N * K * e);
  p.dz = take((bwd || bob) && p.own_dz, T * N * 2 * p.zp);
  p.q = take(bob && p.curved, T * N * 2 * p.zp);
  p.sums = take(bwd || (bob && p.curved), parts * N * 4);
  const size_t f = p.fwd.splits > 1 ? p.fwd.splits * T * N * 4 : 0;
  auto grads = [&](const Splits& n, bool x, bool w) {
    return (x && n.s[0] > 1 ? up(n.s[0] * T * K * 4, ce::kWorkspaceAlign) : 0) +
           (w && n.s[1] > 1 ? up(n.s[1] * (size_t)a.N * K * 4, ce::kWorkspaceAlign) : 0);
  };
  size_t g = 0;
  if (bwd || bob) {
    const size_t each[3] = {grads(p.both, true, true), grads(p.dx, true, false), grads(p.dw, false, true)};
    for (size_t n : each) g = n > g ? n : g;
  }
  p.slab = take(true, pass == LinearPass::kFwd ? f : g);
  p.bytes = at;
  return p;
}

// --- small kernels ---------------------------------------------------------------------------------

// n values of v as np bf16 planes of `stride` elements.
__device__ __forceinline__ void store_planes8(uint16_t* to, size_t stride, int np, float* v) {
  for (int k = 0; k < np; ++k) {
    const uint4 w = bf16x8(v);
    *reinterpret_cast<uint4*>(to + k * stride) = w;
    if (k + 1 == np) break;
    const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // an infinite value has no remainder (inf - inf would make one)
      const float lo = __uint_as_float(h[j] << 16), hi = __uint_as_float(h[j] & 0xffff0000u);
      v[2 * j] = isinf(lo) ? 0.f : v[2 * j] - lo;
      v[2 * j + 1] = isinf(hi) ? 0.f : v[2 * j + 1] - hi;
    }
  }
}

// bf16 planes [np][rows][Kp] of up to four [rows][K] operands in one launch, zero in
// the padding.  One thread per 8 columns; an operand's blocks start at first.
struct Operand {
  const void* x;
  uint16_t* planes;
  long long rows;
  unsigned first;
  int vec;
};
struct Operands {
  Operand o[4];
  int n;
};

template <typename T>
__global__ void __launch_bounds__(256)
    operands_kernel(const __grid_constant__ Operands all, int K, int Kp, int np) {
  allow_next();
  wait_previous();
  int which = 0;
  while (which + 1 < all.n && blockIdx.x >= all.o[which + 1].first) ++which;
  const Operand& o = all.o[which];
  const int per = Kp / 8;
  const long long i = (long long)(blockIdx.x - o.first) * blockDim.x + threadIdx.x, r = i / per;
  const int c = (int)(i - r * per) * 8;
  if (r >= o.rows) return;
  float v[8];
  const T* src = static_cast<const T*>(o.x) + r * K + c;
  if (o.vec)
    load8<T, true>(src, 8, v);
  else
    load8<T, false>(src, K - c, v);
  store_planes8(o.planes + (size_t)r * Kp + c, (size_t)o.rows * Kp, np, v);
}

// dz = m dy a'(z) as np bf16 planes [np][T][Np] (0: not wanted), and its column sums
// per block of `rows_each` rows [parts][Np] (sums may be null).  A warp takes rows of
// 256 columns, a lane eight of them; kDzRows rows are on their way at once, as they
// came: with two, unpacked, the kernel waited for memory (180 us at 8192 x 11,008,
// 100 now).
template <bool SLOPES>
constexpr int kDzRows = SLOPES ? 4 : 8;

template <typename T, bool VEC, bool SLOPES>
__global__ void __launch_bounds__(256, SLOPES ? 2 : 3)
    dz_kernel(const T* dy, const Kept<T>* z, const __grid_constant__ DropArgs da, int act, int rows, int N, int Np,
              int rows_each, uint16_t* planes, int np, float* sums) {
  allow_next();
  wait_previous();
  __shared__ float part[8][256];
  const Dropper drop(da);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + lane * 8;
  const int r0 = blockIdx.y * rows_each, r1 = min(r0 + rows_each, rows);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
  if (c < Np) {
    for (int ra = r0 + warp; ra < r1; ra += 8 * kDzRows<SLOPES>) {
      Raw8<T> g[kDzRows<SLOPES>];
      Raw8<Kept<T>> s[SLOPES ? kDzRows<SLOPES> : 1];
#pragma unroll
      for (int u = 0; u < kDzRows<SLOPES>; ++u) {
        const int r = ra + 8 * u;
        if (r < r1) {
          g[u].template load<VEC>(dy + (size_t)r * N + c, N - c);
          if constexpr (SLOPES) s[u].template load<VEC>(z + (size_t)r * N + c, N - c);
        }
      }
#pragma unroll
      for (int u = 0; u < kDzRows<SLOPES>; ++u) {
        const int r = ra + 8 * u;
        if (r < r1) {
          float v[8];
          g[u].values(v);
          if constexpr (SLOPES) {
            float a1[8];
            s[u].values(a1);
            act_slopes8<sizeof(T) == 4>(act, a1);
            mul8(v, a1);
          }
          if (drop.on) drop.apply8((uint32_t)(c >> 3), (uint32_t)r, v);
          add8(sum, v);
          if (np) store_planes8(planes + (size_t)r * Np + c, (size_t)rows * Np, np, v);
        }
      }
    }
  }
  if (!sums) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = sum[j];
  __syncthreads();
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n < Np) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += part[w][threadIdx.x];
    sums[(size_t)blockIdx.y * Np + n] = t;
  }
}

// What is left when the products are done, in one launch: out [rows][N] = the sum of
// the slabs [splits][rows][Np] of up to two outputs, one thread per 8 columns, with the
// forward's epilogue (FWD); and column sums: col_out [N] = the sum over the parts
// [parts][Np], 32 columns and 8 ways per block, each way and then the ways in order.
struct SlabSum {
  const float* slab;
  void* out;
  long long rows;
  int splits, N, Np, vec;
  unsigned first;  // block
};
struct Finish {
  SlabSum o[2];
  int n;
  unsigned col_first;  // the first block of column sums
  const float* sums;
  void* col_out;
  int parts, col_N, col_Np;
  const void *bias, *r;
  void* z;
  int act;
  DropArgs drop;
};

template <typename T>
__device__ __forceinline__ void sum_parts(const Finish& all) {
  __shared__ float sh[8][32];
  const int x = threadIdx.x & 31, way = threadIdx.x >> 5, n = (int)(blockIdx.x - all.col_first) * 32 + x;
  float s = 0.f;
  if (n < all.col_N) {
    for (int i0 = way; i0 < all.parts; i0 += 8 * 16) {
      float q[16];  // loads first: their latency would be paid one by one
#pragma unroll
      for (int u = 0; u < 16; ++u) q[u] = i0 + 8 * u < all.parts ? all.sums[(size_t)(i0 + 8 * u) * all.col_Np + n] : 0.f;
      float t = 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u) t += q[u];
      s += t;
    }
  }
  sh[way][x] = s;
  __syncthreads();
  if (way != 0 || n >= all.col_N) return;
  s = 0.f;
  for (int w = 0; w < 8; ++w) s += sh[w][x];
  static_cast<T*>(all.col_out)[n] = (T)s;
}

template <typename T, bool FWD>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ Finish all) {
  allow_next();
  wait_previous();
  if (!FWD && blockIdx.x >= all.col_first) return sum_parts<T>(all);
  const SlabSum& o = all.o[all.n > 1 && blockIdx.x >= all.o[1].first];
  const int per = o.Np / 8;
  const long long i = (long long)(blockIdx.x - o.first) * blockDim.x + threadIdx.x, row = i / per;
  const int c = (int)(i - row * per) * 8, n = o.N - c;
  if (row >= o.rows) return;
  const size_t stride = (size_t)o.rows * o.Np, at = (size_t)row * o.Np + c, to = (size_t)row * o.N + c;
  float v[8], w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  for (int s0 = 0; s0 < o.splits; s0 += 4) {
    float f[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s0 + u < o.splits) load8<float, true>(o.slab + (s0 + u) * stride + at, 8, f[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s0 + u < o.splits) add8(v, f[u]);
    }
  }
  T* const out = static_cast<T*>(o.out);
  if constexpr (FWD) {
    const T *bias = static_cast<const T*>(all.bias), *r = static_cast<const T*>(all.r);
    Kept<T>* z = static_cast<Kept<T>*>(all.z);
    if (bias) {
      load8<T, false>(bias + c, n, w);
      add8(v, w);
    }
    if (z) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = sizeof(T) == 2 && all.act == kActRelu ? kept_sign(v[j]) : v[j];
      if (o.vec)
        store8<Kept<T>, true>(z + to, n, w);
      else
        store8<Kept<T>, false>(z + to, n, w);
    }
    act_values8<sizeof(T) == 4>(all.act, v);
    const Dropper drop(all.drop);
    if (drop.on) drop.apply8((uint32_t)(c >> 3), (uint32_t)row, v);
    if (r) {
      if (o.vec)
        load8<T, true>(r + to, n, w);
      else
        load8<T, false>(r + to, n, w);
      add8(v, w);
    }
  }
  if (o.vec)
    store8<T, true>(out + to, n, v);
  else
    store8<T, false>(out + to, n, v);
}

// --- the passes --------------------------------------------------------------------------------------

#define LIN_TRY(x)                    \
  do {                                \
    const cudaError_t e_ = (x);       \
    if (e_ != cudaSuccess) return e_; \
  } while (0)

struct Run {
  const LinearArgs& a;
  const DevCtx& c;
  cudaStream_t s;
  Plan p;
  char* ws;

  template <typename T>
  T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }
  size_t element() const { return a.bf16 ? 2 : 4; }

  template <typename... P, typename... A>
  cudaError_t run(const char* name, void (*kernel)(P...), dim3 grid, dim3 block, A... args) const {
    prof_begin(s, name);
    const cudaError_t e = chained(kernel, grid, block, 0, 1, s, args...);
    prof_end(s);
    return e;
  }

  // Planes of the [.][K] operands that are not read in place.
  cudaError_t operands(const void* x, const void* W, const void* ux, const void* uW) const {
    if (!p.copy_k) return cudaSuccess;
    Operands o;
    o.n = 0;
    long long blocks = 0;
    auto add = [&](const void* v, long long rows, size_t off) {
      if (!v) return;
      o.o[o.n++] = Operand{v, at<uint16_t>(off), rows, (unsigned)blocks, a.K % 8 == 0 && aligned(v, 16)};
      blocks += (rows * (p.Kp / 8) + 255) / 256;
    };
    add(x, a.T, p.x), add(W, a.N, p.W), add(ux, a.T, p.ux), add(uW, a.N, p.uW);
    if (o.n == 0) return cudaSuccess;
    const dim3 grid((unsigned)blocks);
    return a.bf16 ? run("linear_operands", operands_kernel<__nv_bfloat16>, grid, dim3(256), o, a.K, p.Kp, p.np)
                  : run("linear_operands", operands_kernel<float>, grid, dim3(256), o, a.K, p.Kp, p.np);
  }

  void base(GemmArgs& g) const {
    memset(&g, 0, sizeof(g));
    g.fp32 = !a.bf16, g.err = c.err, g.wait_ns = c.wait_ns, g.stall = c.stall;
  }
  static void sizes(Problem& q, long long M, long long N, long long K, int splits) {
    q.M = (int)M, q.N = (int)N, q.K = (int)K, q.splits = splits;
  }
  // Chains of fp32 operands are a stage, so that its small products come before the
  // large ones (chains of two stages: errors of 7e-7 in place of 1.5e-7); long sums of
  // bf16 ones end theirs every 16,384 terms.
  void chains(Problem& q) const {
    const long long terms = ((long long)q.K + q.splits - 1) / q.splits * q.nseg;
    q.chain = !a.bf16 ? 1 : terms > kLongTerms ? (int)(kLongTerms / kBK / q.nseg) : 0;
  }

  // Maps of the planes of a [rows][K] operand, boxes of `box` rows x 64 columns.
  bool maps(CUtensorMap* m, const void* in, size_t off, long long rows, int box) const {
    for (int k = 0; k < p.np; ++k) {
      const void* b = p.copy_k ? at<uint16_t>(off) + (size_t)k * rows * p.Kp : in;
      if (!matrix_map(m + k, b, rows, p.Kp, p.Kp, box)) return false;
    }
    return true;
  }
  // ... of dz (or q): [T][N].  The maps end with the outputs, as those that the epilogue
  // stores through do: what stands in the padding to Np columns is not read (loads fill in zeros).
  bool z_maps(CUtensorMap* m, bool q, int box) const {
    for (int k = 0; k < p.zp; ++k) {
      const void* b = !q && !p.own_dz ? a.dy : at<uint16_t>(q ? p.q : p.dz) + (size_t)k * a.T * p.Np;
      if (!matrix_map(m + k, b, a.T, a.N, p.Np, box)) return false;
    }
    return true;
  }
  bool z_stores(CUtensorMap* m, bool q) const {
    for (int k = 0; k < p.zp; ++k) {
      if (!store_map(m + k, at<uint16_t>(q ? p.q : p.dz) + (size_t)k * a.T * p.Np, a.T, a.N, p.Np)) return false;
    }
    return true;
  }

  // The products of na terms of A operand x and the terms of B operand y (0 or 1
  // each), smallest first; fp32's six share a stage.
  void products(Problem& g, int x, int y, int na) const {
    auto add = [&](int i, int j) { g.seg[g.nseg++] = Seg{(uint8_t)(kPlanes * x + i), (uint8_t)(kPlanes * y + j)}; };
    if (a.bf16) {
      for (int i = na - 1; i >= 0; --i) add(i, 0);
      return;
    }
    add(0, 0);
  }

  bool mapped(const void* t) const { return !t || aligned(t, 16); }

  // y and z from x and W.
  cudaError_t forward() const {
    LIN_TRY(operands(a.x, a.W, nullptr, nullptr));
    GemmArgs g;
    base(g);
    Problem& q = g.prob[0];
    const Shape sh = p.fwd;
    g.problems = 1;
    sizes(q, a.T, a.N, a.K, sh.splits);
    products(q, 0, 0, 1);
    chains(q);
    if (!maps(q.a, a.x, p.x, a.T, 128) || !maps(q.b, a.W, p.W, a.N, sh.tile_n / 2)) return cudaErrorInvalidValue;
    if (sh.splits > 1) {
      q.slab = at<float>(p.slab), q.slab_ld = p.Np;
      LIN_TRY(gemm_slabs(g, s));
      Finish all;
      memset(&all, 0, sizeof(all));
      add_slabs(all, q, a.N, a.y);
      all.bias = a.b, all.r = a.r, all.z = a.z_out, all.act = a.act, all.drop = a.drop;
      all.o[0].vec = all.o[0].vec && mapped(a.r) && mapped(a.z_out);
      return finish(all, true);
    }
    EpArgs& e = g.ep;
    e.bias = a.b, e.in0 = a.r, e.out0 = a.y, e.out1 = a.z_out, e.in_ld = a.N, e.act = a.act, e.drop = a.drop;
    const bool whole = a.bf16 && a.N % 8 == 0;
    e.in_map = whole && mapped(a.r), e.out_map = whole && mapped(a.y) && mapped(a.z_out);
    if (e.in_map && a.r && !store_map(g.in, const_cast<void*>(a.r), a.T, a.N, a.N)) return cudaErrorInvalidValue;
    if (e.out_map && (!store_map(g.out, a.y, a.T, a.N, a.N) ||
                      (a.z_out && !store_map(g.out + 1, a.z_out, a.T, a.N, a.N))))
      return cudaErrorInvalidValue;
    return gemm_forward(sh.tile_n, g, s);
  }

  // The output of a problem whose sums lie in slabs.
  void add_slabs(Finish& all, const Problem& q, int N, void* out) const {
    const int Np = (int)up(N, 8);
    unsigned first = 0;
    if (all.n) first = all.o[0].first + (unsigned)((all.o[0].rows * (all.o[0].Np / 8) + 255) / 256);
    all.o[all.n++] = SlabSum{q.slab, out, q.M, q.splits, N, Np, N % 8 == 0 && aligned(out, 16), first};
  }
  void add_columns(Finish& all, int parts, void* out) const {
    all.sums = at<float>(p.sums), all.col_out = out, all.parts = parts, all.col_N = a.N, all.col_Np = p.Np;
  }
  cudaError_t finish(Finish& all, bool fwd) const {
    unsigned blocks = 0;
    for (int i = 0; i < all.n; ++i) blocks = all.o[i].first + (unsigned)((all.o[i].rows * (all.o[i].Np / 8) + 255) / 256);
    all.col_first = blocks;
    if (all.col_out) blocks += (unsigned)((all.col_N + 31) / 32);
    if (blocks == 0) return cudaSuccess;
    const dim3 grid(blocks), block(256);
    if (a.bf16)
      return run("linear_finish", fwd ? finish_kernel<__nv_bfloat16, true> : finish_kernel<__nv_bfloat16, false>, grid,
                 block, all);
    return run("linear_finish", fwd ? finish_kernel<float, true> : finish_kernel<float, false>, grid, block, all);
  }

  // dz and its column sums out of dy and z.
  cudaError_t make_dz(bool planes, bool sums) const {
    if (!planes && !sums) return cudaSuccess;
    return a.bf16 ? make_dz_as<__nv_bfloat16>(planes, sums) : make_dz_as<float>(planes, sums);
  }
  template <typename E>
  cudaError_t make_dz_as(bool planes, bool sums) const {
    const Kept<E>* z = a.act == kActNone ? nullptr : static_cast<const Kept<E>*>(a.z);
    const bool vec = a.N % 8 == 0 && aligned(a.dy, 16) && mapped(z);
    auto kernel = z ? (vec ? dz_kernel<E, true, true> : dz_kernel<E, false, true>)
                    : (vec ? dz_kernel<E, true, false> : dz_kernel<E, false, false>);
    return run("linear_dz", kernel, dim3((p.Np + 255) / 256, p.sum_parts),
               dim3(256), static_cast<const E*>(a.dy), z, a.drop, a.act, a.T, a.N, p.Np, p.sum_rows,
               at<uint16_t>(p.dz), planes ? p.zp : 0, sums ? at<float>(p.sums) : nullptr);
  }
  // dx [T, K] = q W + dz uW, or (dw) dW [N, K] = q^T x + dz^T ux; either term may be
  // absent (the backward's has dz with the first operand).
  bool gradient(Problem& g, bool dw, int splits, void* out, const void* u, size_t u_off, const void* v,
                size_t v_off) const {
    const long long rows_b = dw ? a.T : a.N;
    sizes(g, dw ? a.N : a.T, a.K, dw ? a.T : a.N, splits);
    g.a_mn = dw;
    const int box_a = dw ? kBK : 128;
    if (u) {  // with q
      if (!z_maps(g.a, true, box_a) || !maps(g.b, u, u_off, rows_b, kBK)) return false;
      products(g, 0, 0, p.zp);
    }
    if (v) {  // with dz
      if (!z_maps(g.a + kPlanes, false, box_a) || !maps(g.b + kPlanes, v, v_off, rows_b, kBK)) return false;
      products(g, 1, 1, p.zp);
    }
    if (g.nseg == 0) return true;
    chains(g);
    g.out0 = out;
    g.out_map = a.bf16 && a.K % 8 == 0 && aligned(out, 16);
    return !g.out_map || store_map(&g.out, out, g.M, a.K, a.K);
  }
  // Both gradients in one launch: u_x, v_x are multiplied by q and dz for dx, u_w, v_w
  // for dW; then what is left, the column sums of `all` among it.
  cudaError_t gradients(Finish& all, const void* u_x, const void* v_x, size_t v_x_off, const void* u_w, const void* v_w,
                        size_t v_w_off) const {
    GemmArgs g;
    base(g);
    const bool want[2] = {a.dx && (u_x || v_x), a.dW && (u_w || v_w)};
    if (a.dx && !want[0]) LIN_TRY(cudaMemsetAsync(a.dx, 0, (size_t)a.T * a.K * element(), s));
    if (a.dW && !want[1]) LIN_TRY(cudaMemsetAsync(a.dW, 0, (size_t)a.N * a.K * element(), s));
    if (!want[0] && !want[1]) return finish(all, false);
    const Splits& n = want[0] && want[1] ? p.both : want[0] ? p.dx : p.dw;
    size_t slab = p.slab;
    // (the order of the slabs in the workspace; the longer tiles' problem is the first of the launch)
    const bool dw_first = want[1] && (!want[0] || steps_of(a.T) / n.s[1] >= steps_of(a.N) / n.s[0]);
    for (int i = 0; i < 2; ++i) {
      if (!want[i]) continue;
      Problem& q = g.prob[want[0] && want[1] ? i != (int)dw_first : 0];
      ++g.problems;
      const bool ok = i ? gradient(q, true, n.s[1], a.dW, u_w, p.x, v_w, v_w_off)
                        : gradient(q, false, n.s[0], a.dx, u_x, p.W, v_x, v_x_off);
      if (!ok) return cudaErrorInvalidValue;
      if (q.splits > 1) {
        q.slab = at<float>(slab), q.slab_ld = p.Kp;
        slab += up((size_t)q.splits * q.M * p.Kp * 4, ce::kWorkspaceAlign);
        add_slabs(all, q, a.K, i ? a.dW : a.dx);
      }
    }
    LIN_TRY(gemm_gradients(g, s));
    return finish(all, false);
  }

  cudaError_t backward() const {
    LIN_TRY(operands(a.dW ? a.x : nullptr, a.dx ? a.W : nullptr, nullptr, nullptr));
    LIN_TRY(make_dz(p.own_dz && (a.dx || a.dW), a.db != nullptr));
    Finish all;
    memset(&all, 0, sizeof(all));
    if (a.db) add_columns(all, p.sum_parts, a.db);
    return gradients(all, nullptr, a.dx ? a.W : nullptr, p.W, nullptr, a.dW ? a.x : nullptr, p.x);
  }

  // dx, dW, db here are gx, gW, gb.
  cudaError_t second() const {
    const bool want_q = p.curved && (a.dx || a.dW || a.db);
    const bool want_dz = (a.dx && a.uW) || (a.dW && a.ux);
    const bool product = a.gdy || want_q;
    Finish all;
    memset(&all, 0, sizeof(all));
    LIN_TRY(operands((product && a.uW) || (want_q && a.dW) ? a.x : nullptr,
                     (product && a.ux) || (want_q && a.dx) ? a.W : nullptr, a.ux, a.uW));
    if (product) {
      GemmArgs g;
      base(g);
      Problem& t = g.prob[0];
      g.problems = 1;
      sizes(t, a.T, a.N, a.K, 1);
      const int box = p.sec.tile_n / 2;
      if (a.ux) {
        if (!maps(t.a, a.ux, p.ux, a.T, 128) || !maps(t.b, a.W, p.W, a.N, box)) return cudaErrorInvalidValue;
        products(t, 0, 0, 1);
      }
      if (a.uW) {
        if (!maps(t.a + kPlanes, a.x, p.x, a.T, 128) || !maps(t.b + kPlanes, a.uW, p.uW, a.N, box))
          return cudaErrorInvalidValue;
        products(t, 1, 1, 1);
      }
      chains(t);
      EpArgs& e = g.ep;
      e.bias = a.ub, e.act = a.act, e.drop = a.drop, e.in_ld = a.N, e.ld = p.Np;
      e.q_planes = want_q && (a.dx || a.dW) ? p.zp : 0;
      e.dz_planes = want_dz && p.own_dz ? p.zp : 0;
      e.sums = want_q && a.db ? at<float>(p.sums) : nullptr;
      e.in0 = a.act == kActNone ? nullptr : a.z;
      e.in1 = want_q || e.dz_planes ? a.dy : nullptr;
      e.out0 = a.gdy;
      const bool whole = a.bf16 && a.N % 8 == 0;
      e.in_map = whole && mapped(e.in0) && mapped(e.in1), e.out_map = whole && mapped(a.gdy);
      if (e.in_map && ((e.in0 && !store_map(g.in, const_cast<void*>(e.in0), a.T, a.N, a.N)) ||
                       (e.in1 && !store_map(g.in + 1, const_cast<void*>(e.in1), a.T, a.N, a.N))))
        return cudaErrorInvalidValue;
      if (e.out_map && a.gdy && !store_map(g.out, a.gdy, a.T, a.N, a.N)) return cudaErrorInvalidValue;
      if ((e.q_planes && !z_stores(g.out + 2, true)) || (e.dz_planes && !z_stores(g.out + 2 + kPlanes, false)))
        return cudaErrorInvalidValue;
      LIN_TRY(gemm_second(p.sec.tile_n, g, s));
      if (e.sums) add_columns(all, (a.T + 31) / 32, a.db);
    } else if (want_dz && p.own_dz) {
      LIN_TRY(make_dz(true, false));
    }
    if (a.db && !p.curved) LIN_TRY(cudaMemsetAsync(a.db, 0, a.N * element(), s));
    const bool q = p.curved;
    return gradients(all, q ? a.W : nullptr, a.uW, p.uW, q ? a.x : nullptr, a.ux, p.ux);
  }
};

}  // namespace
}  // namespace lin

bool linear_is_plain(const LinearArgs& a, LinearPass pass) {
  return pass == LinearPass::kFwd && lin::takes_rows(a);
}

size_t linear_workspace(const LinearArgs& a, LinearPass pass) {
  if (linear_is_plain(a, pass)) return 0;
  const size_t n = lin::plan(a, pass).bytes;
  return n ? n + ce::kWorkspaceSlack : 0;
}

cudaError_t linear(const LinearArgs& a, LinearPass pass, const DevCtx& c, cudaStream_t s) {
  if (linear_is_plain(a, pass)) return lin::rows(a, s);
  const lin::Run r{a, c, s, lin::plan(a, pass), static_cast<char*>(ce::workspace_base(a.ws))};
  switch (pass) {
    case LinearPass::kFwd: return r.forward();
    case LinearPass::kBwd: return r.backward();
    case LinearPass::kBob: return r.second();
  }
  return cudaErrorInvalidValue;
}

}  // namespace fbob
