// Internal interface of the linear head's cross entropy: the tensor-core
// product kernel (ce_gemm.cu) and the passes that call it (linear_ce.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace fbob {
namespace ce {

constexpr int kTileM = 256;     // rows of a pair's tile (128 per block)
constexpr int kTileN = 256;     // columns of a tile with one accumulator
constexpr int kTileNDual = 128; // ... with two
constexpr int kBK = 64;         // contraction per stage (128 bytes of bf16)
constexpr int kPlanes = 3;      // bf16 terms that stand for one fp32 operand
constexpr int kMaxMaps = 2 * kPlanes;
constexpr int kMaxSegs = 2 * 6;
// bf16 operands: up to this many counted tokens G and Z keep two bf16 terms.  The
// second ones have room for that many tokens' rows (whole steps) only.
constexpr int kExactTokens = 16;
constexpr int kLowRows = kBK;

// A product's operands: planes are bf16 matrices, a segment multiplies plane a
// by plane b; the sum over the segments is the product.  With two accumulators
// a segment stands for z += a[a] b[b] and b += a[kPlanes + a] b[b] +
// a[a] b[kPlanes + b] (each term only if its second-order operand is there).
struct Seg {
  uint8_t a, b;
};

// What becomes of an accumulator tile.
enum Epilogue {
  kStats,   // row maxima and sums of exponentials per 128 columns, target logits
  kGrad,    // G = gs (p - onehot) as bf16 planes
  kAlpha,   // (two accumulators z, b) row sums of p b
  kGrad2,   // (two accumulators) Z = gs p (b - alpha) and G, as bf16 planes
  kSlab,    // fp32, optionally added to what is there
  kOut      // scaled, in the output type
};

struct EpArgs {
  // tokens (kStats .. kGrad2): rows of the tile, counted tokens only
  const int* index;       // [T]: the caller's row of each counted token
  const int* target;      // [T]: its column
  const float* lse;       // [T], the caller's rows
  const float* g;         // [T], the caller's rows
  const float* gmax;      // [1]: gs = g / gmax
  const float* alpha;     // [T]
  float2* part;           // kStats: (max, sum) [parts][T], two parts per tile of columns
  float* sums;            // kAlpha: row sums [parts][T], two parts per tile of columns
  float* picked;          // kStats: [T], z at the target
  // kSlab, kOut
  void* out;
  long long out_ld, slab;  // elements between rows, between split slabs
  int accumulate, out_bf16, out_map;  // out_map: bf16 results leave through GemmArgs::c[0]
};

struct GemmArgs {
  CUtensorMap a[kMaxMaps], b[kMaxMaps];
  CUtensorMap c[kMaxMaps];  // store_map()s: kGrad, kGrad2: G planes, then Z planes; kOut: the output
  Seg seg[kMaxSegs];
  int nseg, nlow;       // the first nlow are left out if more than kExactTokens tokens count
  int fp32;             // operands stand for fp32 (kPlanes planes, sums kept to fp32)
  int has_ua, has_ub;   // two accumulators: which second-order operands are there
  int K;                // contraction length
  int splits;           // K is cut into at most this many slabs (kSlab)
  const int* slabs;     // the number wanted, on the device (kSlab)
  int M, N;             // output rows and columns
  // The counted tokens lie in the first *count of T rows.  They are the rows of
  // kStats .. kSlab (M = T at most) and the contraction of kOut (K = T at most);
  // kGrad and kGrad2 also write zero rows up to token_steps() x 64, which kOut
  // reads.
  const int* count;
  int n_base;           // kStats..kGrad2: vocabulary index of column 0
  int b0;               // offset into the rows of the matrices B is read from
  EpArgs ep;
  unsigned int* err;
  unsigned long long wait_ns;
  int stall;
};

// The slabs are read and written 32 bytes at a time and every part of the plan
// starts a multiple of 256 bytes after the workspace's base.  Callers' workspaces
// are 16-byte aligned, so the base is the next 256-byte bound; the slack for it
// is part of the size that callers are told.
constexpr size_t kWorkspaceAlign = 256;
constexpr size_t kWorkspaceSlack = kWorkspaceAlign - 16;
inline void* workspace_base(void* ws) {
  return reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + kWorkspaceAlign - 1) & ~(uintptr_t)(kWorkspaceAlign - 1));
}

// Rows, in steps of the contraction, that hold n counted tokens (at least one
// step, so that a sum over no tokens is written as zero).
__host__ __device__ inline int token_steps(int n) { return n <= kBK ? 1 : (n + kBK - 1) / kBK; }

// Sums of kSlab and kOut over K terms of each of nseg segments (those of low
// terms not counted: 2^-8 of the others, they come first, while the accumulator is
// as small).  Above 16,384 terms in all a chain of the tensor cores ends after
// long_chain() steps of every segment, again 16,384 terms.
constexpr int kLongTerms = 16384;
__host__ __device__ inline int long_chain(int nseg) { return kLongTerms / kBK / nseg; }
__host__ __device__ inline bool long_sum(int K, int nseg) { return (long long)K * nseg > kLongTerms; }

// C = sum over segments of A_seg B_seg^T with A [M][K], B [N][K], then the
// epilogue.  kSlab reads B and kOut reads both A and B from matrices stored
// with the contraction outermost ([K][N], [K][M]).
cudaError_t gemm(Epilogue ep, const GemmArgs& g, cudaStream_t s);

// 2-D map of a bf16 matrix [rows][cols] with `ld` elements per row and a box
// of box_rows x 64 columns, 128-byte swizzle.
bool matrix_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box_rows);

// The same matrix as the epilogue stores it: boxes of 32 x 32, 64-byte swizzle.
bool store_map(CUtensorMap* m, void* base, long long rows, long long cols, long long ld);

}  // namespace ce
}  // namespace fbob
