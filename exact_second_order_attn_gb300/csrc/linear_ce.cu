// Softmax cross entropy of a linear head z = h W^T over a large vocabulary,
// without keeping the logits: forward, gradients, and the gradients' own
// vector-Jacobian product (formulas in fbob.h).
//
// Tokens that are not counted cost nothing: a first kernel lists the others, and
// every product works on the listed rows only (their number stays on the
// device; launches are sized for all tokens, blocks without tiles end at once).
//
// Forward: one product whose epilogue reduces each 128 columns of a row to
// (max, sum of exponentials) and picks the target's logit; a small kernel joins
// them.  Gradients: for pieces of the vocabulary, the logits are formed again
// and turned in the epilogue into G = (g / gmax) (p - onehot), kept as bf16 for
// the piece only; then dH += G W and dW = gmax G^T H.  Second order: one pass
// for alpha = sum p b, then the same with Z = (g / gmax) p (b - alpha) beside G.
//
// Dividing by gmax = max |g| (an fp32 factor of the results) keeps the target's
// entry of G at p - 1 for a mean loss, where all g are equal: its rounding to
// bf16 is then relative to p - 1 and not a systematic relative error of the
// largest entry of every row.  With unequal g it is one: against 64 bits dH and dW
// are 1.34 times as far off as a result that is rounded once (rows 2.7 times at
// most; 1.01 and 1.65 with equal g; 24 to 4096 tokens x 8000 classes x 768, g of
// 0.1 to 1), what a gradient of the logits kept in bf16 costs.  A second term of G
// for every token would cost two more products beside the step's four.  The
// roundings average out over many tokens; with few a row of dW hangs on one or two
// of them (4 tokens: 1.6 times the error of a result rounded once; 24: 1.05 times),
// so up to kExactTokens counted ones G and Z keep two bf16 terms (2^-17): 14 us of
// 127 at 24 tokens x 50,257 classes x 768.  How many count is known on the device,
// so the kernels choose.
//
// Measured: 8192 tokens (a tenth ignored) x 50,257 classes x 768, bf16, forward
// and gradients 1.40 ms in a burst (1.60 ms under the power cap), 4096 with the
// second order 2.65 (2.77) ms; 24 tokens 109 us, bound by reading and writing W
// and dW and by ten launches; fp32 1021 x 32,003 x 512 610 us.
//
// fp32 inputs stand as three bf16 terms each (8 bits of the value per term);
// the six products of terms whose magnitudes reach 2^-16 of the first are
// summed, smallest first, in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "ce.h"
#include "launch.cuh"
#include "prof.h"

namespace fbob {
namespace ce {
namespace {

constexpr int kPairs = 76;                        // block pairs of a GB300, for the split rule
constexpr size_t kPieceBytes = 512ull << 20;      // G (and Z) of one piece of the vocabulary
constexpr size_t kPieceLeast = 2048;              // columns, whatever they take
constexpr int kPieceStep = 256;

size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// bf16 planes of G and of Z, and the rows that plane k has room for.
int grad_planes(const CeArgs& a) { return a.bf16 ? 2 : kPlanes; }
long long plane_rows(const CeArgs& a, int k) { return a.bf16 && k > 0 && a.T > kLowRows ? kLowRows : a.T; }
long long plane_rows_to(const CeArgs& a, int k) {  // of the planes before k
  long long n = 0;
  for (int i = 0; i < k; ++i) n += plane_rows(a, i);
  return n;
}

// Piece width: all of V if its G fits kPieceBytes, else equal pieces that do, or
// of 2048 columns where fewer would fit: dW has a tile of rows per 256 columns, and
// fewer leave the device idle (262,144 tokens x 8192 classes x 768, backward: 54 ms
// with 256 columns, 15.6 with 1024, 9.4 with 2048, 6.9 with 4096).
int piece_cols(const CeArgs& a, bool second) {
  // (kLowRows rows beside more tokens' are not counted: 128 bytes of a class)
  const size_t rows = a.bf16 && a.T > kLowRows ? a.T : plane_rows_to(a, grad_planes(a));
  const size_t per = rows * 2 * (second ? 2 : 1);
  size_t cols = a.piece > 0 ? (size_t)a.piece : kPieceBytes / (per ? per : 1);
  cols = up(cols < kPieceLeast && a.piece <= 0 ? kPieceLeast : cols, kPieceStep);
  const size_t whole = up(a.V, kPieceStep);
  if (cols >= whole) return (int)whole;
  const size_t n = (a.V + cols - 1) / cols;
  return (int)up((a.V + n - 1) / n, kPieceStep);
}

// Slabs of the contraction over a piece in dH = G W.  Its output has few tiles
// (counted tokens x D), so the contraction is cut until the tiles' last wave is
// nearly full; each slab costs a write and a read of T x D floats.  How many
// tokens count is known on the device only: the host bounds the number (256 MB
// of slabs, and at least eight 64-class steps in each), the list kernel chooses.
int most_slabs(const CeArgs& a, int cols) {
  const size_t slab = (size_t)a.T * up(a.D, 8) * 4;
  const size_t room = (256u << 20) / (slab ? slab : 1), steps = up(cols, kBK) / kBK / 8;
  const size_t most = room < steps ? room : steps;
  return most < 1 ? 1 : most > 64 ? 64 : (int)most;
}

// What the list kernel finds out: counted tokens, gmax and slabs of dH.
struct Totals {
  int count;
  float gmax;
  int slabs;
};

// Where everything lies in the workspace.
struct Plan {
  int np, gp, Dp, ld, splits, stat_parts, alpha_parts;
  bool copy_w;
  size_t h, uh, w, uw, place, index, target, totals, part, sums, picked, alpha, planes, slab, bytes;
};

Plan plan(const CeArgs& a, CePass pass) {
  Plan p;
  p.np = a.bf16 ? 1 : kPlanes;
  p.gp = grad_planes(a);
  p.Dp = (int)up(a.D, 8);
  p.copy_w = !a.bf16 || a.D % 8 != 0;
  p.stat_parts = 2 * ((a.V + kTileN - 1) / kTileN);
  p.alpha_parts = 2 * ((a.V + kTileNDual - 1) / kTileNDual);
  p.ld = pass == CePass::kFwd ? 0 : piece_cols(a, pass == CePass::kBob);
  p.splits = pass == CePass::kFwd ? 1 : most_slabs(a, p.ld);
  size_t at = 0;
  auto take = [&](bool want, size_t bytes) {
    const size_t here = at;
    if (want) at += up(bytes, kWorkspaceAlign);
    return here;
  };
  const bool bwd = pass != CePass::kFwd, bob = pass == CePass::kBob;
  const size_t T = a.T, V = a.V, row = (size_t)p.Dp * 2 * p.np;
  p.h = take(true, T * row);
  p.uh = take(bob, T * row);
  p.w = take(p.copy_w, V * row);
  p.uw = take(bob && p.copy_w, V * row);
  p.place = take(true, T * 4);
  p.index = take(true, T * 4);
  p.target = take(true, T * 4);
  p.totals = take(true, sizeof(Totals));
  p.picked = take(!bwd, T * 4);
  p.part = take(!bwd, T * p.stat_parts * sizeof(float2));
  p.sums = take(bob, T * p.alpha_parts * 4);
  p.alpha = take(bob, T * 4);
  p.planes = take(bwd, (size_t)plane_rows_to(a, p.gp) * p.ld * 2 * (bob ? 2 : 1));
  p.slab = take(bwd, T * p.Dp * 4 * p.splits);
  p.bytes = at;
  return p;
}

// --- small kernels ---------------------------------------------------------------------------------

// The counted tokens, in order: index[i] is the caller's row of the i-th one and
// target[i] its column; place[r] is that i for row r, -1 if it is ignored, -2 if
// its target is outside the vocabulary (reported in the status word).  Also
// gmax = max |g| over them (1 if that is not finite).  One block: 8192 tokens
// per round, a prefix sum over the warps' counts.
constexpr int kListThreads = 1024, kListItems = 8;

__global__ void __launch_bounds__(kListThreads)
    list_kernel(const long long* target, const float* g, long long ignore, int V, int T, int* place, int* index,
                int* column, Totals* totals, int D, int most, unsigned int* err) {
  allow_next();
  wait_previous();
  __shared__ int warp_n[32];
  __shared__ float warp_m[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = 0.f;
  int before = 0;  // counted tokens of the earlier rounds
  bool wrong = false;
  for (int t0 = 0; t0 < T; t0 += kListThreads * kListItems) {
    // item i of this thread: row i of the 32-token rows of its warp
    const int first = t0 + warp * 32 * kListItems + lane;
    long long y[kListItems];
    float w[kListItems];
    unsigned kept[kListItems];
    int n = 0;  // counted tokens of the warp
#pragma unroll
    for (int i = 0; i < kListItems; ++i) {
      const int t = first + 32 * i;
      y[i] = t < T ? target[t] : ignore;
      w[i] = g && t < T ? fabsf(g[t]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kListItems; ++i) {
      const bool keep = y[i] != ignore && y[i] >= 0 && y[i] < V;
      wrong |= !keep && y[i] != ignore;
      if (keep) m = fmaxf(m, w[i]);
      kept[i] = __ballot_sync(0xffffffffu, keep);
      n += __popc(kept[i]);
    }
    if (lane == 0) warp_n[warp] = n;
    __syncthreads();
    int mine = lane < warp ? warp_n[lane] : 0, all = warp_n[lane];  // of the warps before, of all
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mine += __shfl_xor_sync(0xffffffffu, mine, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    int at = before + mine;
#pragma unroll
    for (int i = 0; i < kListItems; ++i) {
      const int t = first + 32 * i;
      const bool keep = kept[i] >> lane & 1u;
      const int to = at + __popc(kept[i] & ((1u << lane) - 1u));
      if (t < T) place[t] = keep ? to : y[i] == ignore ? -1 : -2;
      if (keep) {
        index[to] = t;
        column[to] = (int)y[i];
      }
      at += __popc(kept[i]);
    }
    before += all;
    __syncthreads();
  }
  if (wrong) atomicOr(err, kErrTarget);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) warp_m[warp] = m;
  __syncthreads();
  if (warp == 0) {
    m = warp_m[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // slabs: the fewest that fill the waves to 93 %, else those that fill them best
    const int tiles = max(1, (before + kTileM - 1) / kTileM) * ((D + kTileN - 1) / kTileN);
    float best = 0.f;
    int slabs = 1;
    for (int s = lane + 1; s <= most; s += 32) {
      const long long n = (long long)tiles * s;
      const float full = fminf((float)n / (float)((n + kPairs - 1) / kPairs * kPairs), 0.93f);
      if (full > best) best = full, slabs = s;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float full = __shfl_xor_sync(0xffffffffu, best, o);
      const int s = __shfl_xor_sync(0xffffffffu, slabs, o);
      if (full > best || (full == best && s < slabs)) best = full, slabs = s;
    }
    if (lane == 0) *totals = Totals{before, m < INFINITY ? m : 1.f, slabs};
  }
}

// bf16 planes [np][rows][Dp] of up to four operands in one launch: of the counted
// rows of H and UH (then zero rows up to a whole step of the contraction), and of
// W and UW where they are not read in place; zero in the padding.  One thread per
// 8 columns; an operand's blocks start at first_block.
struct Operand {
  const void* x;
  uint16_t* planes;
  long long rows;
  unsigned first_block;
  int tokens, vec;
};
struct Operands {
  Operand o[4];
  int n;
};

template <typename T>
__global__ void __launch_bounds__(256)
    planes_kernel(const __grid_constant__ Operands all, const int* index, const Totals* totals, int D, int Dp, int np) {
  allow_next();
  wait_previous();
  int which = 0;
  while (which + 1 < all.n && blockIdx.x >= all.o[which + 1].first_block) ++which;
  const Operand& o = all.o[which];
  const long long rows = o.rows;
  uint16_t* const planes = o.planes;
  const bool vec = o.vec;
  const int per = Dp / 8;
  const long long i = (long long)(blockIdx.x - o.first_block) * blockDim.x + threadIdx.x;
  const long long r = i / per;
  const int c = (int)(i - r * per) * 8;
  if (r >= rows) return;
  const int count = o.tokens ? totals->count : 0;
  if (o.tokens && r >= (long long)token_steps(count) * kBK) return;
  float v[8];
  if (o.tokens && r >= count) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  } else {
    const T* src = static_cast<const T*>(o.x) + (o.tokens ? index[r] : r) * D + c;
    if (vec) {
      if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      } else {
        const float4 f = *reinterpret_cast<const float4*>(src), g = *reinterpret_cast<const float4*>(src + 4);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w, v[4] = g.x, v[5] = g.y, v[6] = g.z, v[7] = g.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = c + j < D ? (float)src[j] : 0.f;
    }
  }
  for (int k = 0; k < np; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
      // an infinite value has no remainder (inf - inf would make one)
      const float2 f = __bfloat1622float2(h);
      v[2 * j] = isinf(f.x) ? 0.f : v[2 * j] - f.x;
      v[2 * j + 1] = isinf(f.y) ? 0.f : v[2 * j + 1] - f.y;
    }
    *reinterpret_cast<uint4*>(planes + ((size_t)k * rows + r) * Dp + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Sums over `parts` per-row partials, 32 rows per block, 16 threads per row:
// loss and lse (kStats), or alpha and gg (kAlpha).
constexpr int kJoinRows = 32, kJoinWays = 16, kJoinLoads = 8;

__global__ void __launch_bounds__(kJoinRows* kJoinWays)
    join_stats_kernel(const float2* part, int parts, const int* place, const float* picked, int T, float* loss,
                      float* lse) {
  allow_next();
  wait_previous();
  __shared__ float2 sh[kJoinWays][kJoinRows];
  const int t = blockIdx.x * kJoinRows + threadIdx.x;
  const int at = t < T ? place[t] : -1;
  float m = -INFINITY, s = 0.f;
  if (at >= 0) {
    for (int i0 = threadIdx.y; i0 < parts; i0 += kJoinWays * kJoinLoads) {
      float2 q[kJoinLoads];  // loads first: their latency would be paid one by one
      float top = m;
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) {
        const int i = i0 + u * kJoinWays;
        q[u] = i < parts ? part[(size_t)i * T + at] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) top = fmaxf(top, q[u].x);
      if (m > -INFINITY) s *= expf(m - top);
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) s += q[u].x > -INFINITY ? q[u].y * expf(q[u].x - top) : q[u].y;
      m = top;
    }
  }
  sh[threadIdx.y][threadIdx.x] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.y != 0 || t >= T) return;
  float top = -INFINITY;
  for (int w = 0; w < kJoinWays; ++w) top = fmaxf(top, sh[w][threadIdx.x].x);
  s = 0.f;
  for (int w = 0; w < kJoinWays; ++w) {
    const float2 q = sh[w][threadIdx.x];
    s += q.x > -INFINITY ? q.y * expf(q.x - top) : q.y;
  }
  const float l = (top > -INFINITY ? top : 0.f) + logf(s);
  lse[t] = at >= 0 ? l : 0.f;
  loss[t] = at >= 0 ? l - picked[at] : at == -1 ? 0.f : NAN;
}

// alpha, and gg = alpha - b at the target, with b's row summed here in fp32
// (one warp per token): out of the tensor cores' chain it would carry 1e-6.
template <typename T>
__global__ void __launch_bounds__(kJoinRows* kJoinWays)
    join_alpha_kernel(const float* sums, int parts, const int* place, const int* column, const T* H, const T* W,
                      const T* UH, const T* UW, int T_, int D, float* alpha, float* gg) {
  allow_next();
  wait_previous();
  __shared__ float sh[kJoinWays][kJoinRows];
  __shared__ float total[kJoinRows];
  const int t = blockIdx.x * kJoinRows + threadIdx.x;
  const int at = t < T_ ? place[t] : -1;
  float s = 0.f;
  if (at >= 0) {
    for (int i0 = threadIdx.y; i0 < parts; i0 += kJoinWays * kJoinLoads) {
      float q[kJoinLoads];
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) {
        const int i = i0 + u * kJoinWays;
        q[u] = i < parts ? sums[(size_t)i * T_ + at] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kJoinLoads; ++u) s += q[u];
    }
  }
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0) {
    s = 0.f;
    for (int w = 0; w < kJoinWays; ++w) s += sh[w][threadIdx.x];
    total[threadIdx.x] = s;
    if (at >= 0) alpha[at] = s;
  }
  __syncthreads();
  if (!gg) return;
  for (int i = threadIdx.y; i < kJoinRows; i += kJoinWays) {
    const int r = blockIdx.x * kJoinRows + i;
    if (r >= T_) break;
    const int from = place[r];
    float b = 0.f;
    if (from >= 0) {
      const int y = column[from];
#pragma unroll 4
      for (int c = threadIdx.x; c < D; c += 32) {
        if (UH) b += (float)UH[(size_t)r * D + c] * (float)W[(size_t)y * D + c];
        if (UW) b += (float)H[(size_t)r * D + c] * (float)UW[(size_t)y * D + c];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
    if (threadIdx.x == 0) gg[r] = from >= 0 ? total[i] - b : 0.f;
  }
}

// out [T][D] = gmax * sum of the slabs [T][Dp]; zero in rows that are not counted.
template <typename T>
__global__ void __launch_bounds__(256)
    finish_kernel(const float* slab, long long stride, const int* place, const Totals* totals, T* out,
                  int D, int Dp, long long rows, int vec) {
  allow_next();
  wait_previous();
  const int per = Dp / 4;
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long r = i / per;
  const int c = (int)(i - r * per) * 4;
  if (r >= rows) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  const int at = place[r];
  if (at >= 0) {
    const float gm = totals->gmax;
    const int splits = totals->slabs;
    for (int s0 = 0; s0 < splits; s0 += 8) {
      float4 f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        f[u] = s0 + u < splits ? *reinterpret_cast<const float4*>(slab + (s0 + u) * stride + (long long)at * Dp + c)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < 8; ++u) v[0] += f[u].x, v[1] += f[u].y, v[2] += f[u].z, v[3] += f[u].w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= gm;
  }
  if (c >= D) return;  // the slabs' padding
  T* o = out + r * D + c;
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(o) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c + j < D) o[j] = (T)v[j];
    }
  }
}

// --- the passes --------------------------------------------------------------------------------------

#define CE_TRY(x)                                \
  do {                                           \
    const cudaError_t e_ = (x);                  \
    if (e_ != cudaSuccess) return e_;            \
  } while (0)

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

struct Run {
  const CeArgs& a;
  const DevCtx& c;
  cudaStream_t s;
  Plan p;
  char* ws;
  bool second;

  template <typename T>
  T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }

  // The list of counted tokens, and H, W (UH, UW) as the products read them.
  cudaError_t operands() const {
    prof_begin(s, "ce_list");
    const cudaError_t e = chained(list_kernel, dim3(1), dim3(kListThreads), 0, 1, s, a.target, a.g, a.ignore, a.V, a.T,
                                  at<int>(p.place), at<int>(p.index), at<int>(p.target), at<Totals>(p.totals), a.D,
                                  p.splits, c.err);
    prof_end(s);
    CE_TRY(e);
    Operands o;
    o.n = 0;
    long long blocks = 0;
    auto add = [&](const void* x, bool tokens, size_t off) {
      if (!x) return;
      const long long rows = tokens ? a.T : a.V;
      o.o[o.n++] = Operand{x, at<uint16_t>(off), rows, (unsigned)blocks, tokens, a.D % 8 == 0 && aligned(x, 16)};
      blocks += (rows * (p.Dp / 8) + 255) / 256;
    };
    add(a.H, true, p.h);
    if (second) add(a.UH, true, p.uh);
    if (p.copy_w) add(a.W, false, p.w);
    if (p.copy_w && second) add(a.UW, false, p.uw);
    prof_begin(s, "ce_operands");
    const cudaError_t f = a.bf16 ? chained(planes_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(256), 0, 1, s, o,
                                           at<int>(p.index), at<Totals>(p.totals), a.D, p.Dp, p.np)
                                 : chained(planes_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, 1, s, o,
                                           at<int>(p.index), at<Totals>(p.totals), a.D, p.Dp, p.np);
    prof_end(s);
    return f;
  }

  GemmArgs base() const {
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    g.splits = 1, g.fp32 = !a.bf16;
    g.err = c.err, g.wait_ns = c.wait_ns, g.stall = c.stall;
    g.count = &at<Totals>(p.totals)->count, g.slabs = &at<Totals>(p.totals)->slabs;
    g.ep.index = at<int>(p.index), g.ep.target = at<int>(p.target), g.ep.lse = a.lse, g.ep.g = a.g;
    g.ep.gmax = &at<Totals>(p.totals)->gmax;
    return g;
  }

  // Maps of the planes of a [rows][D] operand (of the tokens, or of the head).
  bool token_maps(CUtensorMap* m, size_t off, int box) const {
    for (int k = 0; k < p.np; ++k)
      if (!matrix_map(m + k, at<uint16_t>(off) + (size_t)k * a.T * p.Dp, a.T, p.Dp, p.Dp, box)) return false;
    return true;
  }
  bool head_maps(CUtensorMap* m, const void* x, size_t off, int box) const {
    for (int k = 0; k < p.np; ++k) {
      const void* b = p.copy_w ? at<uint16_t>(off) + (size_t)k * a.V * p.Dp : x;
      if (!matrix_map(m + k, b, a.V, p.Dp, p.Dp, box)) return false;
    }
    return true;
  }
  // Planes of G (which = 0) or Z (1) of a piece of `cols` columns.
  uint16_t* piece_plane(int which, int k) const {
    return at<uint16_t>(p.planes) + (size_t)(which * plane_rows_to(a, p.gp) + plane_rows_to(a, k)) * p.ld;
  }
  bool piece_maps(CUtensorMap* m, int which, int cols, int box) const {
    for (int k = 0; k < p.gp; ++k)
      if (!matrix_map(m + k, piece_plane(which, k), plane_rows(a, k), cols, p.ld, box)) return false;
    return true;
  }

  // The products of the terms of A operand `x` and B operand `y` (0 or 1 each),
  // np of each, that reach 2^-16 of the first, smallest first.
  void products(GemmArgs& g, int x, int y) const {
    for (int order = p.np - 1; order >= 0; --order) {
      for (int i = order; i >= 0; --i)
        g.seg[g.nseg++] = Seg{(uint8_t)(kPlanes * x + i), (uint8_t)(kPlanes * y + order - i)};
    }
  }
  // The same with A operands of pieces: G (x = 0), or Z (1) and, with an operand
  // of its own, G.  The second terms of bf16's G and Z go first.
  void piece_products(GemmArgs& g, bool both) const {
    const int xs[2] = {second ? 1 : 0, 0}, n = both ? 2 : 1;
    for (int i = 0; i < n && p.np < p.gp; ++i) {
      g.seg[g.nseg++] = Seg{(uint8_t)(kPlanes * xs[i] + 1), (uint8_t)(kPlanes * i)};
      ++g.nlow;
    }
    for (int i = 0; i < n; ++i) products(g, xs[i], i);
  }

  // The logits (and, in the second order, b = UH W^T + H UW^T).
  bool logits(GemmArgs& g, bool dual) const {
    const int box = (dual ? kTileNDual : kTileN) / 2;
    if (!token_maps(g.a, p.h, 128) || !head_maps(g.b, a.W, p.w, box)) return false;
    products(g, 0, 0);
    if (dual) {
      if (a.UH && !token_maps(g.a + kPlanes, p.uh, 128)) return false;
      if (a.UW && !head_maps(g.b + kPlanes, a.UW, p.uw, box)) return false;
      g.has_ua = a.UH != nullptr, g.has_ub = a.UW != nullptr;
    }
    g.M = a.T, g.K = a.D;
    return true;
  }

  cudaError_t stats() const {
    GemmArgs g = base();
    if (!logits(g, false)) return cudaErrorInvalidValue;
    g.N = a.V;
    g.ep.part = at<float2>(p.part), g.ep.picked = at<float>(p.picked);
    CE_TRY(gemm(kStats, g, s));
    prof_begin(s, "ce_join");
    const cudaError_t e = chained(join_stats_kernel, dim3((a.T + kJoinRows - 1) / kJoinRows),
                                  dim3(kJoinRows, kJoinWays), 0, 1, s, at<float2>(p.part), p.stat_parts,
                                  at<int>(p.place), at<float>(p.picked), a.T, a.loss, a.lse_out);
    prof_end(s);
    return e;
  }

  cudaError_t alpha() const {
    GemmArgs g = base();
    if (!logits(g, true)) return cudaErrorInvalidValue;
    g.N = a.V;
    g.ep.sums = at<float>(p.sums);
    CE_TRY(gemm(kAlpha, g, s));
    prof_begin(s, "ce_join");
    const cudaError_t e = a.bf16 ? join_alpha<__nv_bfloat16>() : join_alpha<float>();
    prof_end(s);
    return e;
  }
  template <typename E>
  cudaError_t join_alpha() const {
    return chained(join_alpha_kernel<E>, dim3((a.T + kJoinRows - 1) / kJoinRows), dim3(kJoinRows, kJoinWays), 0, 1, s,
                   at<float>(p.sums), p.alpha_parts, at<int>(p.place), at<int>(p.target), static_cast<const E*>(a.H),
                   static_cast<const E*>(a.W), static_cast<const E*>(a.UH), static_cast<const E*>(a.UW), a.T, a.D,
                   at<float>(p.alpha), a.gg);
  }

  // One piece of the vocabulary: columns c0 .. c0 + cols - 1.
  cudaError_t piece(int c0, int cols, bool first) const {
    GemmArgs g = base();
    if (!logits(g, second)) return cudaErrorInvalidValue;
    g.N = cols, g.n_base = g.b0 = c0;
    g.ep.alpha = at<float>(p.alpha);
    for (int k = 0; k < p.gp; ++k) {
      const long long rows = plane_rows(a, k);
      if (!store_map(g.c + k, piece_plane(0, k), rows, cols, p.ld)) return cudaErrorInvalidValue;
      if (second && !store_map(g.c + kPlanes + k, piece_plane(1, k), rows, cols, p.ld)) return cudaErrorInvalidValue;
    }
    CE_TRY(gemm(second ? kGrad2 : kGrad, g, s));
    if (a.dH) {  // Z W + G UW, or G W
      g = base();
      if (!piece_maps(g.a, 0, cols, 128) || !head_maps(g.b, a.W, p.w, 64)) return cudaErrorInvalidValue;
      if (second) {
        if (!piece_maps(g.a + kPlanes, 1, cols, 128)) return cudaErrorInvalidValue;
        if (a.UW && !head_maps(g.b + kPlanes, a.UW, p.uw, 64)) return cudaErrorInvalidValue;
      }
      piece_products(g, second && a.UW);
      g.M = a.T, g.N = a.D, g.K = cols, g.b0 = c0;
      // every slab gets at least one step: a short last piece adds to the first slabs only
      const int steps = (cols + kBK - 1) / kBK;
      g.splits = p.splits < steps ? p.splits : steps;
      g.ep.out = at<float>(p.slab), g.ep.out_ld = p.Dp, g.ep.slab = (long long)a.T * p.Dp, g.ep.accumulate = !first;
      CE_TRY(gemm(kSlab, g, s));
    }
    if (a.dW) {  // Z^T H + G^T UH, or G^T H
      g = base();
      if (!piece_maps(g.a, 0, cols, 64) || !token_maps(g.b, p.h, 64)) return cudaErrorInvalidValue;
      if (second) {
        if (!piece_maps(g.a + kPlanes, 1, cols, 64)) return cudaErrorInvalidValue;
        if (a.UH && !token_maps(g.b + kPlanes, p.uh, 64)) return cudaErrorInvalidValue;
      }
      piece_products(g, second && a.UH);
      g.M = cols, g.N = a.D, g.K = a.T;
      g.ep.out = static_cast<char*>(a.dW) + (size_t)c0 * a.D * (a.bf16 ? 2 : 4);
      g.ep.out_ld = a.D, g.ep.out_bf16 = a.bf16;
      // bulk stores want 16-byte rows; a piece's rows end with a tile's, or with W's
      g.ep.out_map = a.bf16 && a.D % 8 == 0 && aligned(a.dW, 16);
      if (g.ep.out_map && !store_map(g.c, g.ep.out, cols, a.D, a.D)) return cudaErrorInvalidValue;
      CE_TRY(gemm(kOut, g, s));
    }
    return cudaSuccess;
  }

  cudaError_t finish() const {
    if (!a.dH) return cudaSuccess;
    prof_begin(s, "ce_finish");
    const cudaError_t e = a.bf16 ? finish_as<__nv_bfloat16>() : finish_as<float>();
    prof_end(s);
    return e;
  }
  template <typename E>
  cudaError_t finish_as() const {
    const long long n = (long long)a.T * (p.Dp / 4);
    const int vec = a.D % 4 == 0 && aligned(a.dH, 4 * sizeof(E));
    return chained(finish_kernel<E>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, 1, s, at<float>(p.slab),
                   (long long)a.T * p.Dp, at<int>(p.place), at<Totals>(p.totals), static_cast<E*>(a.dH), a.D, p.Dp,
                   (long long)a.T, vec);
  }
};

}  // namespace
}  // namespace ce

size_t linear_ce_workspace(const CeArgs& a, CePass pass) { return ce::plan(a, pass).bytes + ce::kWorkspaceSlack; }

cudaError_t linear_ce(const CeArgs& a, CePass pass, const DevCtx& c, cudaStream_t s) {
  const ce::Run r{a, c, s, ce::plan(a, pass), static_cast<char*>(ce::workspace_base(a.ws)),
                  pass == CePass::kBob};
  CE_TRY(r.operands());
  if (pass == CePass::kFwd) return r.stats();
  if (pass == CePass::kBob) CE_TRY(r.alpha());
  if (!a.dH && !a.dW) return cudaSuccess;
  for (int c0 = 0; c0 < a.V; c0 += r.p.ld)
    CE_TRY(r.piece(c0, a.V - c0 < r.p.ld ? a.V - c0 : r.p.ld, c0 == 0));
  return r.finish();
}

}  // namespace fbob
