// Internal interface of linear layers: the tensor-core product kernel
// (linear_gemm.cuh), the product of a few tokens (linear_rows.cu) and the passes
// that call them (linear.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace fbob {
namespace lin {

constexpr int kTileM = 256;  // rows of a pair's tile (128 per block)
constexpr int kBK = 64;      // contraction per stage (128 bytes of bf16)
constexpr int kPlanes = 3;   // bf16 terms that stand for one fp32 operand
constexpr int kMaxSegs = 4;
// bf16 operands: up to this many tokens dz and q keep two bf16 terms.
constexpr int kExactTokens = 16;

// A segment multiplies plane a by plane b (fp32: the planes from a and b on, the six
// products that count); the sum over the segments is the product.
struct Seg {
  uint8_t a, b;
};

// How A [M, K] and B [N, K] are stored.
enum Layout {
  kNT,         // A [M][K], B [N][K]
  kGradients,  // A [M][K] (dz for dx) or [K][M] (dz for dW), B [K][N]
};
// What becomes of an accumulator tile.
enum Epilogue {
  kForward,      // y = r + m a(v + bias), and z = v + bias
  kSecond,       // v + bias = t: gdy, q, dz and q's column sums; one term of q and dz
  kSecondTerms,  // the same with several (tiles of 128 columns)
  kGradient,     // in the output type, or a slab
  kSlab          // fp32
};

struct EpArgs {
  const void *bias;         // [N], or null
  const void *in0, *in1;    // kForward: r, -; kSecond: z, dy (null: absent)
  void *out0, *out1;        // kForward: y, z; kSecond: gdy (null: not wanted)
  float* sums;              // kSecond: column sums of q [rows / 32][ld], or null
  long long ld, in_ld;      // of the sums; of the inputs and outputs (elements)
  int in_map, out_map;      // inputs and outputs move through the maps (bf16)
  int q_planes, dz_planes;  // bf16 terms of q and dz (0: not wanted), stored through out[2], out[5]
  int act;
  DropArgs drop;
};

struct Problem {
  CUtensorMap a[2 * kPlanes], b[2 * kPlanes];
  CUtensorMap out;  // store_map() of out0
  Seg seg[kMaxSegs];
  int nseg, a_mn;
  int M, N, K, splits;
  int chain;          // steps of K after which a chain of the tensor cores ends (0: never)
  int out_map;        // results leave through the map (bf16)
  void* out0;         // kGradient: [M][N]
  float* slab;        // or [splits][M][slab_ld]
  long long slab_ld;
};

struct GemmArgs {
  Problem prob[2];
  CUtensorMap in[2];                 // store_map()s of in0, in1
  CUtensorMap out[2 + 2 * kPlanes];  // of out0, out1, q's planes, dz's planes
  int problems, fp32;
  int stages, boxes;  // of a block, of an epilogue warp: set at the launch
  EpArgs ep;
  unsigned int* err;
  unsigned long long wait_ns;
  int stall;
};

// C = sum over segments of A_seg B_seg^T, then the epilogue; tiles of kTileM x
// tile_n (128, 192 or 256).  Splits are at most the steps of K.
cudaError_t gemm_forward(int tile_n, const GemmArgs& g, cudaStream_t s);  // kNT, kForward
cudaError_t gemm_second(int tile_n, const GemmArgs& g, cudaStream_t s);   // kNT, kSecond or kSecondTerms
cudaError_t gemm_slabs(const GemmArgs& g, cudaStream_t s);                // kNT, kSlab
cudaError_t gemm_gradients(const GemmArgs& g, cudaStream_t s);            // kGradients, kGradient

// y (and z) of up to kRowsTokens tokens without tensor cores (linear_rows.cu, which has
// the times of both ways).  For bf16 the tiles are as fast on the GPU from 2^25 products on,
// from 2^26.5 where they need a copy of W (rows that are no multiples of 16 bytes), but a call
// costs the host 8.9 us against 3.8: the bounds are 2^26 and 2^27 (1024 -> 4096, 16 tokens,
// 12.2 us here and 7.9 in tiles).  One token never is.  fp32 tiles read W in three terms: they
// are as fast from some 2^29 products, 12 tokens of the widest layers, which is left to the rows.
constexpr int kRowsTokens = 16;
inline bool takes_rows(const LinearArgs& a) {
  if (a.T <= 1) return true;
  return a.T <= kRowsTokens && (!a.bf16 || (long long)a.T * a.K * a.N <= 1ll << (a.K % 8 ? 27 : 26));
}
cudaError_t rows(const LinearArgs& a, cudaStream_t s);

}  // namespace lin
}  // namespace fbob
