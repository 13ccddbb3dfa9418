// The matrix products of the linear head's cross entropy on the fifth
// generation tensor cores, with the softmax work in the epilogue.
//
// C[256 x 256] = sum over segments of A_seg B_seg^T per pair of thread blocks
// (cta_group::2): each block holds its 128 rows of A and its half of B's rows
// of every 64-column stage, so a stage moves 32 KB per block for
// 128 x 256 x 64 products, half of what a lone block would read from L2; the
// accumulator's 128 rows x 256 columns lie in the block's tensor memory, two
// of them, so the epilogue of one tile runs under the products of the next.
// The kernels with two accumulators (z and b of the second order) use 128
// columns each, and their stages hold both operands of both sides (48 KB for
// three products of 128 x 128 x 64, the same traffic per product).
//
// The tensor cores drop the bits of a step's sum below the accumulator's last
// one, an error that grows with the chain of steps (4e-6 of the result at 32,000
// terms).  That is too much for fp32 operands, and for the fp32 results of bf16
// ones (losses, alpha: 1e-6 to 4e-6 at D above 500).  There a chain ends after
// kChainBlocks stages of each plane product (bf16: 512 columns) and the epilogue
// threads add the chains up in registers, rounding to nearest.  Shorter chains cost
// time and longer ones bits (D = 768: 256 columns 20 % of these kernels' time, 512
// 6 %, the whole width 2 %; of drawn cases of all widths 0.06, 0.09 and 0.7 % are
// further off than 1e-6 and 1.5 times an fp32 sum).  The gradients' sums, which
// are rounded to bf16, run over tokens or classes without limit: where those are
// more than 16,384, both products of the second order counted, their chains end
// there (1,024 steps, 3e-5; shorter sums keep the plain epilogue, 10 us of 119 at
// 24 tokens).  G, rounded to bf16, has one chain over D.
//
// Roles of a block's eleven warps: 0-7 epilogue (thread = accumulator row, the
// two warpgroups take half of the columns each), 8 and 10 TMA producers of A and
// of B (one warp for both: G kernel 3 % slower), 9 MMA issue (the
// leader block's) and TMEM allocation.  Barriers: full[s] of the leader counts
// both blocks' bytes; empty[s] and tile_full[b] are signalled in both blocks
// by the MMAs' commit; tile_empty[b] of the leader counts the 16 epilogue
// warps of the pair.  Every wait is bounded.  Blocks are persistent: pair i
// takes tiles i, i + pairs, ...; tiles walk over 8 row tiles per column tile,
// so that both operands are re-read from L2.
//
// Measured on 7,373 counted tokens x 50,257 classes x 768 (569 GFLOP a product,
// burst clock): logits with statistics 332 us (1,710 TFLOP/s), with G 350, G W 353,
// G^T H 312 us; half as many tokens, alpha's three products 563 us.  Bound by the
// tensor cores; a tile of K = 768 in one chain takes 6,900 cycles where its MMAs
// need 6,144, since stages come at 64 bytes per cycle and multiprocessor.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>

#include "ce.h"
#include "launch.cuh"
#include "prof.h"
#include "tc_pair.cuh"

namespace fbob {
namespace ce {
namespace {

using namespace tc;

constexpr int kThreads = 352;
constexpr int kEpWarps = 8;
constexpr int kGroupM = 8;        // row tiles per raster group
constexpr int kTmemCols = 512;
constexpr int kBufCols = 256;     // accumulator columns per tile in flight
constexpr uint64_t kDrainNs = 200000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kBoxBytes = 32 * 32 * 2;  // an outgoing box: a warp's 32 rows x 32 columns of bf16
// Whether a tile's contraction is cut into chains that are added up in
// registers, and the chains' length in steps of 64 columns.
// LONG: kSlab and kOut of bf16 operands where long_sum(); chains of long_chain().
template <int EP, bool FP32, bool LONG>
constexpr bool kHeld = FP32 || LONG || EP == kStats || EP == kAlpha;
template <bool FP32>
constexpr int kChainBlocks = FP32 ? 2 : 8;

template <int EP>
struct Cfg {
  static constexpr bool DUAL = EP == kAlpha || EP == kGrad2;
  static constexpr bool A_MN = EP == kOut;
  static constexpr bool B_MN = EP == kSlab || EP == kOut;
  static constexpr int BN = DUAL ? kTileNDual : kTileN;
  static constexpr int A_BYTES = 128 * kBK * 2;
  static constexpr int B_BYTES = BN / 2 * kBK * 2;
  static constexpr int STAGE = (A_BYTES + B_BYTES) * (DUAL ? 2 : 1);  // [A | B], or [A | UA | B | UB]
  static constexpr int NST = 196608 / STAGE;  // 6, or 4 with two accumulators
  static constexpr int OUT_OFF = NST * STAGE;  // the epilogue warps' outgoing boxes
  static constexpr int SMEM = OUT_OFF + kEpWarps * 2 * kBoxBytes;
  static_assert(SMEM + 1024 <= 232448, "shared memory budget");
};

struct Ctrl {
  uint64_t full[8], empty[8], tile_full[2], tile_empty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};

// A wait whose arrivals may come from the other block of the cluster (with
// mbar_arrive_relaxed).
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, const Waiter& w) {
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (try_wait_cluster(bar, parity)) return true;
    if ((it & 15u) == 0u) {
      if (*w.abort) return false;
      if (globaltimer_ns() - t0 > w.limit) {
        *w.abort = 1;
        atomicOr(w.err, kErrTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^(z - at) for the softmax: the difference is taken first, so that its
// rounding is relative to it and not to the logit.  For bf16 operands the
// special function unit's 2^x of a rounded product (error about 5e-7 at
// z - at = -15) is far below the rounding of G; fp32 operands take expf.
template <bool FP32>
__device__ __forceinline__ float ex(float z, float at) {
  return FP32 ? expf(z - at) : ex2((z - at) * kLog2e);
}

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// An epilogue warp's way out for bf16 results: 32 rows x 32 columns (lane =
// row) go to shared memory with the 64-byte swizzle and leave as one bulk tensor
// store, clipped at the matrix's ends (a box starts inside it); two boxes take
// turns.  Stored from the
// registers, a row per lane, the same bytes cost the load-store unit 32 lines
// per instruction and bound the G kernel (8,300 of 8,800 cycles per tile).
struct Outbox {
  uint32_t smem;  // this warp's two boxes
  int turn;
  __device__ __forceinline__ void put(const CUtensorMap* map, int x, int y, const uint32_t (&w)[16]) {
    const uint32_t lane = threadIdx.x & 31, box = smem + turn * kBoxBytes;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();  // the box's earlier content has left
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c)
      st_shared_v4(box + lane * 64 + ((c ^ ((lane >> 1) & 3u)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                   w[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      asm volatile(
          "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
          "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
          "r"(box), "r"(x), "r"(y)
          : "memory");
    }
    turn ^= 1;
  }
  // Everything has been written (the lane that issued the stores).
  __device__ __forceinline__ void drain() const {
    if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
};

// 32 values as bf16 planes (n of them, or kPlanes): plane k holds the rounding of
// what planes 0..k-1 left.
template <bool FP32>
__device__ __forceinline__ void store_planes(Outbox& out, const CUtensorMap* maps, int n, int x, int y, float* v) {
  // (fp32 unrolled; bf16 has one plane, two where few tokens count)
#pragma unroll(FP32 ? kPlanes : 1)
  for (int k = 0; k < (FP32 ? kPlanes : n); ++k) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      const float2 f = __bfloat1622float2(h);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
      v[2 * j] -= f.x;
      v[2 * j + 1] -= f.y;
    }
    out.put(maps + k, x, y, w);
  }
}

// 32 columns of an accumulator, from tensor memory or from the registers in
// which its chains were added up (c is then a constant: unrolled loops).
template <bool HELD>
struct Acc {
  uint32_t tmem;
  const float* sum;
  uint32_t freed;  // the leader's tile_empty barrier of this accumulator
  __device__ __forceinline__ void load(int tmem_col, int at, float* v) const {
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = sum[at + j];
    } else {
      __syncwarp();  // the load is warp-collective, the code between loads is not
      tmem_ld32(tmem + tmem_col, v);
    }
  }
  // The warp has read its part: the accumulator may be written again.
  __device__ __forceinline__ void done() const {
    if constexpr (!HELD) {
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive_relaxed(freed);
    }
  }
};

// The epilogue of one tile for this thread's row: `row` in the output, n0 the
// first column, part the index of this half tile's row statistics.
template <int EP, bool FP32, bool HELD>
__device__ __forceinline__ void epilogue(const GemmArgs& p, const Acc<HELD>& acc, Outbox& out, int rows, int row, int n0,
                                         int part, int split, bool few) {
  constexpr int W = Cfg<EP>::BN / 2, kUnroll = HELD ? 4 : 1;  // columns of this thread (of each accumulator)
  const EpArgs& e = p.ep;
  const bool live = row < rows;
  const int box_row = row - (int)(threadIdx.x & 31);  // of the warp's first row
  const int planes = !FP32 && few && box_row < kLowRows ? 2 : 1;  // of bf16 G and Z
  if constexpr (EP == kStats) {
    const int y = live ? e.target[row] : -1;
    float m = -INFINITY, s = 0.f;
#pragma unroll kUnroll
    for (int c = 0; c < W; c += 32) {
      float v[32];
      acc.load(c, c, v);
      if (c + 32 == W) acc.done();
      const int n = n0 + c;
      if (y >= n && y < n + 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (n + j == y) e.picked[row] = v[j];
        }
      }
      if (n + 32 > p.N) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = n + j < p.N ? v[j] : -INFINITY;
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < 32; ++j) top = fmaxf(top, v[j]);
      if (top > -INFINITY || top != top) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) t += ex<FP32>(v[j], top);
        s = s * ex<FP32>(m, top) + t;
        m = top;
      } else {  // nothing above -inf so far; a NaN among them still counts
#pragma unroll
        for (int j = 0; j < 32; ++j) s += v[j] != v[j] ? v[j] : 0.f;
      }
    }
    if (live) e.part[(size_t)part * p.M + row] = make_float2(m, s);
  } else if constexpr (EP == kGrad) {
    const int y = live ? e.target[row] : -1, own = live ? e.index[row] : 0;
    const float at = live ? e.lse[own] : 0.f, gm = *e.gmax;
    const float gs = live && gm != 0.f ? e.g[own] / gm : 0.f;
#pragma unroll kUnroll
    for (int c = 0; c < W; c += 32) {
      float v[32];
      acc.load(c, c, v);
      if (c + 32 == W) acc.done();
      const int n = n0 + c, hit = y - p.n_base - n;
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = live ? gs * ex<FP32>(v[j], at) : 0.f;
      if (live && hit >= 0 && hit < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] -= j == hit ? gs : 0.f;
      }
      if (box_row < p.M && n < p.N) store_planes<FP32>(out, p.c, planes, n, box_row, v);  // rows past the tokens: zero
    }
  } else if constexpr (EP == kAlpha) {
    const float at = live ? e.lse[e.index[row]] : 0.f;
    float s = 0.f;
#pragma unroll kUnroll
    for (int c = 0; c < W; c += 32) {
      float z[32], b[32];
      acc.load(c, c, z);
      acc.load(kTileNDual + c, W + c, b);
      if (c + 32 == W) acc.done();
      const int n = n0 + c;
#pragma unroll
      for (int j = 0; j < 32; ++j) s += n + j < p.N ? ex<FP32>(z[j], at) * b[j] : 0.f;
    }
    if (live) e.sums[(size_t)part * p.M + row] = s;
  } else if constexpr (EP == kGrad2) {
    const int y = live ? e.target[row] : -1, own = live ? e.index[row] : 0;
    const float at = live ? e.lse[own] : 0.f, al = live ? e.alpha[row] : 0.f, gm = *e.gmax;
    const float gs = live && gm != 0.f ? e.g[own] / gm : 0.f;
#pragma unroll kUnroll
    for (int c = 0; c < W; c += 32) {
      float z[32], b[32];
      acc.load(c, c, z);
      acc.load(kTileNDual + c, W + c, b);
      if (c + 32 == W) acc.done();
      const int n = n0 + c, hit = y - p.n_base - n;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        z[j] = live ? gs * ex<FP32>(z[j], at) : 0.f;
        b[j] = live ? z[j] * (b[j] - al) : 0.f;
      }
      if (live && hit >= 0 && hit < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] -= j == hit ? gs : 0.f;
      }
      if (box_row < p.M && n < p.N) {  // rows past the tokens: zero
        store_planes<FP32>(out, p.c, planes, n, box_row, z);
        store_planes<FP32>(out, p.c + kPlanes, planes, n, box_row, b);
      }
    }
  } else if constexpr (EP == kSlab) {
    float* slab = static_cast<float*>(e.out) + (size_t)split * e.slab + (size_t)row * e.out_ld;
#pragma unroll kUnroll
    for (int c = 0; c < W; c += 32) {
      float v[32];
      acc.load(c, c, v);
      if (c + 32 == W) acc.done();
      const int n = n0 + c;
#pragma unroll
      for (int j = 0; j < 32; j += 8) {  // out_ld is a multiple of 8
        if (live && n + j < e.out_ld) {
          float* o = slab + n + j;
          if (e.accumulate) {
            const float4 h = *reinterpret_cast<const float4*>(o), i = *reinterpret_cast<const float4*>(o + 4);
            v[j] += h.x, v[j + 1] += h.y, v[j + 2] += h.z, v[j + 3] += h.w;
            v[j + 4] += i.x, v[j + 5] += i.y, v[j + 6] += i.z, v[j + 7] += i.w;
          }
          st_global_v8(o, reinterpret_cast<const uint32_t*>(v + j));
        }
      }
    }
  } else {
    const float gm = *e.gmax;
    const size_t at = (size_t)row * e.out_ld;
#pragma unroll kUnroll
    for (int c = 0; c < W; c += 32) {
      float v[32];
      acc.load(c, c, v);
      if (c + 32 == W) acc.done();
      const int n = n0 + c;
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= gm;
      if (!FP32 && e.out_map) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        if (box_row < p.M && n < p.N) out.put(p.c, n, box_row, w);
      } else if (!live) {
      } else if (e.out_bf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(e.out) + at + n;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (n + j < p.N) o[j] = __float2bfloat16_rn(v[j]);
        }
      } else {
        float* o = static_cast<float*>(e.out) + at + n;
        const bool whole = (reinterpret_cast<uintptr_t>(e.out) & 31) == 0 && e.out_ld % 8 == 0;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          if (whole && n + j + 8 <= p.N) {
            st_global_v8(o + j, reinterpret_cast<const uint32_t*>(v + j));
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              if (n + j + q < p.N) o[j + q] = v[j + q];
            }
          }
        }
      }
    }
  }
}

// Fewer than 2^31 tiles (the sizes are checked): 32-bit arithmetic throughout,
// since a division of 64 bits costs the issuing threads more than a product.
struct Tiles {
  int mt, nt, splits, kb;  // row and column tiles, slabs, 64-column steps of K
  __device__ __forceinline__ int count() const { return mt * nt * splits; }
  __device__ __forceinline__ int split(int i) const { return splits == 1 ? 0 : i / (mt * nt); }
  __device__ __forceinline__ void at(int i, int& m, int& n) const {
    const int r = splits == 1 ? i : i % (mt * nt);
    const int first = r / (kGroupM * nt) * kGroupM;
    const int in = r - first * nt, rows = min(kGroupM, mt - first);
    n = in / rows;
    m = first + in - n * rows;
  }
  __device__ __forceinline__ int k_first(int split) const {
    return splits == 1 ? split * kb : (int)((long long)kb * split / splits);
  }
};

// A place in the ring of stages and its pass over the ring.
template <int NST>
struct Place {
  int s = 0;
  uint32_t pass = 0;
  __device__ __forceinline__ void next() {
    if (++s == NST) s = 0, pass ^= 1;
  }
};

template <int EP, bool FP32, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs p) {
  using C = Cfg<EP>;
  constexpr bool HELD = kHeld<EP, FP32, LONG>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Ctrl ctrl;
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  allow_next();

  if (tid == 0) {
    ctrl.abort_flag = 0;
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&ctrl.full[s], 1);
      mbar_init(&ctrl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl.tile_full[b], 1);
      mbar_init(&ctrl.tile_empty[b], 2 * kEpWarps);
    }
    mbar_init(&ctrl.drain, 1);
    fence_mbar_init();
    if ((smem_u32(smem) & 1023u) != 0u) {
      ctrl.abort_flag = 1;
      atomicOr(p.err, kErrTimeout);
    }
  }
  if (warp == 9) {
    tmem_alloc_pair(&ctrl.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers are initialised
  tc_fence_after();
  const uint32_t tb = ctrl.tmem_base;
  const Waiter wt{&ctrl.abort_flag, p.err, p.wait_ns};
  const bool live = ctrl.abort_flag == 0;
  const uint32_t sm0 = smem_u32(smem);
  wait_previous();
  const int tokens = *p.count, written = min(p.M, token_steps(tokens) * kBK);
  const int rows = EP == kOut ? p.M : tokens;                             // that hold results
  const int tile_rows = EP == kGrad || EP == kGrad2 ? written : rows;     // that are worked on
  const bool few = tokens <= kExactTokens;
  const int seg0 = few ? 0 : p.nlow;
  const Tiles ts{(tile_rows + kTileM - 1) / kTileM, (p.N + C::BN - 1) / C::BN, EP == kSlab ? min(p.splits, *p.slabs) : 1,
                 EP == kOut ? token_steps(tokens) : (p.K + kBK - 1) / kBK};
  const int total = ts.count(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  // the steps of K up to which an accumulator chain that starts at kc runs
  const int chain_steps = LONG ? long_chain(p.nseg - p.nlow) : kChainBlocks<FP32>;
  auto chain_end = [chain_steps](int kc, int k1) { return HELD ? min(kc + chain_steps, k1) : k1; };

  if (warp == 8 || warp == 10) {
    // ------------------------------------------- TMA: warp 8 loads A, warp 10 loads B
    const bool is_a = warp == 8;
    if (live) {  // the whole warp runs the loop; one lane issues (elect.sync)
      const uint32_t full0 = map_rank(smem_u32(&ctrl.full[0]), 0);
      const uint32_t stage_bytes = 2 * (C::DUAL ? C::A_BYTES * (1 + p.has_ua) + C::B_BYTES * (1 + p.has_ub) : C::STAGE);
      Place<C::NST> at;
      long long issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        int m, n;
        ts.at(t, m, n);
        const int split = ts.split(t);
        const int row = m * kTileM + (int)rank * 128, col = n * C::BN + (int)rank * (C::BN / 2);
        const int k0 = ts.k_first(split), k1 = ts.k_first(split + 1);
        for (int kc = k0; ok && kc < k1; kc = chain_end(kc, k1)) {
          const int ke = chain_end(kc, k1);
          for (int s = seg0; ok && s < p.nseg; ++s) {
            const CUtensorMap* ma = &p.a[p.seg[s].a];
            const CUtensorMap* mb = &p.b[p.seg[s].b];
            for (int k = kc; k < ke; ++k, ++issued, at.next()) {
              const int st = at.s;
              if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.empty[st], at.pass ^ 1, wt)))) break;
              if (p.stall && issued == 0) continue;  // test hook: nothing fills the first stage
              const uint32_t bar = full0 + 8 * st;
              const uint32_t da = sm0 + st * C::STAGE, db = da + (C::DUAL ? 2 : 1) * C::A_BYTES;
              if (is_a) {
                if (rank == 0) mbar_expect_tx_w(&ctrl.full[st], stage_bytes);
                if (C::A_MN) {
                  tma_load_2d_pair(da, ma, bar, row, k * kBK);
                  tma_load_2d_pair(da + 8192, ma, bar, row + 64, k * kBK);
                } else {
                  tma_load_2d_pair(da, ma, bar, k * kBK, row);
                }
                if (C::DUAL && p.has_ua) tma_load_2d_pair(da + C::A_BYTES, ma + kPlanes, bar, k * kBK, row);
              } else {
                if (C::B_MN) {
                  tma_load_2d_pair(db, mb, bar, col, p.b0 + k * kBK);
                  tma_load_2d_pair(db + 8192, mb, bar, col + 64, p.b0 + k * kBK);
                } else {
                  tma_load_2d_pair(db, mb, bar, k * kBK, p.b0 + col);
                }
                if (C::DUAL && p.has_ub) tma_load_2d_pair(db + C::B_BYTES, mb + kPlanes, bar, k * kBK, p.b0 + col);
              }
            }
          }
        }
      }
      // The last use of each stage: on the leader its loads have landed, in both
      // blocks the MMAs' arrivals have (on the give-up path after a limit), so
      // nothing is in flight towards a block that has ended.
      for (long long i = issued > C::NST ? issued - C::NST : 0; i < issued; ++i) {
        const int st = (int)(i % C::NST);
        if (rank == 0 && !ok) mbar_wait_drain(&ctrl.full[st], (i / C::NST) & 1, kDrainNs);
        if (ok) ok = mbar_wait(&ctrl.empty[st], (i / C::NST) & 1, wt);
      }
      if (!ok && rank != 0) {  // this block's loads count on the leader's barriers: give them time to land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kDrainNs) {
        }
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ MMA
    if (live && rank == 0) {
      constexpr uint32_t id = idesc_bf16(kTileM, C::BN, C::A_MN, C::B_MN);
      constexpr uint32_t lbo_a = C::A_MN ? 8192 : 16, lbo_b = C::B_MN ? 8192 : 16;
      constexpr uint32_t step_a = C::A_MN ? 2048 >> 4 : 32 >> 4, step_b = C::B_MN ? 2048 >> 4 : 32 >> 4;
      Place<C::NST> at;
      int chain = 0;  // accumulator buffers handed to the epilogue so far
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const int split = ts.split(t);
        const int k0 = ts.k_first(split), k1 = ts.k_first(split + 1);
        for (int kc = k0; ok && kc < k1; kc = chain_end(kc, k1), ++chain) {
          const int ke = chain_end(kc, k1), buf = chain & 1;
          ok = __all_sync(0xffffffffu, wait_cluster(&ctrl.tile_empty[buf], ((chain >> 1) & 1) ^ 1, wt));
          tc_fence_after();
          const uint32_t d = tb + buf * kBufCols;
          for (int s = seg0; ok && s < p.nseg; ++s) {
            for (int k = kc; k < ke; ++k, at.next()) {
              const int st = at.s;
              ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.full[st], at.pass, wt));
              if (!ok) break;
              tc_fence_after();
              const uint32_t more = s > seg0 || k > kc;  // the accumulator holds a product already
              const uint32_t a = desc_lo(sm0 + st * C::STAGE, lbo_a);
              const uint32_t b = desc_lo(sm0 + st * C::STAGE + (C::DUAL ? 2 : 1) * C::A_BYTES, lbo_b);
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk)
                mma_ss_pair(d, a + kk * step_a, b + kk * step_b, id, kk > 0 ? 1u : more);
              if (C::DUAL) {
                if (p.has_ua) {
#pragma unroll
                  for (int kk = 0; kk < kBK / 16; ++kk)
                    mma_ss_pair(d + kTileNDual, a + (C::A_BYTES >> 4) + kk * step_a, b + kk * step_b, id,
                                kk > 0 ? 1u : more);
                }
                if (p.has_ub) {
#pragma unroll
                  for (int kk = 0; kk < kBK / 16; ++kk)
                    mma_ss_pair(d + kTileNDual, a + kk * step_a, b + (C::B_BYTES >> 4) + kk * step_b, id,
                                kk > 0 ? 1u : more | p.has_ua);
                }
              }
              mma_commit_pair(&ctrl.empty[st]);
            }
          }
          mma_commit_pair(&ctrl.tile_full[buf]);
        }
      }
      mma_commit_pair(&ctrl.drain);  // the last MMA has read its operands
      mbar_wait_drain(&ctrl.drain, 0, kDrainNs);
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int half = warp >> 2, r = (warp & 3) * 32 + (tid & 31);
    const uint32_t lane = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t freed = map_rank(smem_u32(&ctrl.tile_empty[0]), 0);
    Outbox out{sm0 + C::OUT_OFF + warp * 2 * kBoxBytes, 0};
    int chain = 0;
    bool ok = live;
    for (int t = pair; ok && t < total; t += pairs) {
      int m, n;
      ts.at(t, m, n);
      const int split = ts.split(t);
      constexpr int H = C::BN / 2;
      const int row = m * kTileM + (int)rank * 128 + r, n0 = n * C::BN + half * H;
      if constexpr (HELD) {
        float sum[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) sum[j] = 0.f;
        const int k0 = ts.k_first(split), k1 = ts.k_first(split + 1);
        for (int kc = k0; kc < k1; kc = chain_end(kc, k1), ++chain) {
          const int buf = chain & 1;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.tile_full[buf], (chain >> 1) & 1, wt)))) break;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[32];
            // two accumulators: 64 columns of each
            tmem_ld32(tb + lane + buf * kBufCols + half * H + (C::DUAL ? (q >> 1) * kTileNDual + (q & 1) * 32 : q * 32), v);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[q * 32 + j] += v[j];
          }
          tc_fence_before();
          __syncwarp();
          if ((tid & 31) == 0) mbar_arrive_relaxed(freed + buf * 8);
        }
        if (ok) epilogue<EP, FP32, true>(p, Acc<true>{0, sum, 0}, out, rows, row, n0, 2 * n + half, split, few);
      } else {
        const int buf = chain & 1;
        // warp-uniform: the TMEM loads that follow are warp-collective
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.tile_full[buf], (chain >> 1) & 1, wt)))) break;
        tc_fence_after();
        epilogue<EP, FP32, false>(p, Acc<false>{tb + lane + buf * kBufCols + half * H, nullptr, freed + buf * 8}, out, rows, row, n0, 2 * n + half,
                            split, few);
        ++chain;
      }
    }
    out.drain();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither block ends, or frees tensor memory, before the other is done
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tb, kTmemCols);
  }
}

template <int EP, bool FP32, bool LONG>
cudaError_t launch_as(const GemmArgs& g, const char* name, cudaStream_t s) {
  using C = Cfg<EP>;
  auto kernel = gemm_kernel<EP, FP32, LONG>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((g.M + kTileM - 1) / kTileM) * ((g.N + C::BN - 1) / C::BN) * g.splits;
  if (tiles == 0) return cudaSuccess;
  const long long pairs = sm_count() / 2;
  prof_begin(s, name);
  e = chained(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kThreads), C::SMEM, 2, s, g);
  prof_end(s);
  return e;
}

template <int EP>
cudaError_t launch(const GemmArgs& g, const char* name, cudaStream_t s) {
  if (g.fp32) return launch_as<EP, true, false>(g, name, s);
  if constexpr (EP == kSlab || EP == kOut) {
    if (long_sum(g.K, g.nseg - g.nlow)) return launch_as<EP, false, true>(g, name, s);
  }
  return launch_as<EP, false, false>(g, name, s);
}

}  // namespace

cudaError_t gemm(Epilogue ep, const GemmArgs& g, cudaStream_t s) {
  switch (ep) {
    case kStats: return launch<kStats>(g, "ce_stats", s);
    case kGrad: return launch<kGrad>(g, "ce_grad", s);
    case kAlpha: return launch<kAlpha>(g, "ce_alpha", s);
    case kGrad2: return launch<kGrad2>(g, "ce_grad2", s);
    case kSlab: return launch<kSlab>(g, "ce_hidden", s);
    case kOut: return launch<kOut>(g, "ce_head", s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace ce
}  // namespace fbob
