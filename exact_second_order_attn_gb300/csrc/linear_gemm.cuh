// The matrix products of linear layers on the fifth generation tensor cores, with
// the layer's elementwise work in the epilogue.
//
// C[256 x BN] = sum over segments of A_seg B_seg^T per pair of thread blocks
// (cta_group::2): each block holds its 128 rows of A and its half of B's rows of
// every 64-column stage; the accumulator's 128 rows x BN columns lie in the block's
// tensor memory, two of them, so the epilogue of one tile runs under the products
// of the next.
//
// fp32 operands are three bf16 terms each, and the six products of terms that reach
// 2^-16 of the first are summed, smallest first.  The tensor cores drop the bits of
// a step's sum below the accumulator's last one, so there a chain ends after 128
// columns and the epilogue threads add the chains up in registers (HELD); so do sums
// of bf16 operands over more than 16,384 terms, every 16,384 (3e-5 of the result).
//
// Roles of a block's eleven warps: 0-7 epilogue (thread = accumulator row, the two
// warpgroups take half of the columns each), 8 and 10 TMA producers of A and of B, 9
// MMA issue (the leader block's) and TMEM allocation.  Barriers: full[s] of the
// leader counts both blocks' bytes; empty[s] and tile_full[b] are signalled in both
// blocks by the MMAs' commit; tile_empty[b] of the leader counts the 16 epilogue
// warps of the pair.  Every wait is bounded.  Blocks are persistent: pair i takes
// tiles i, i + pairs, ...
//
// What the epilogue reads beside the accumulator (the residual; z and dy of the
// second order) comes in boxes of a warp's 32 rows x 32 columns: bulk tensor loads
// two boxes ahead, which run under the products of the tile that the warp waits for;
// results leave in such boxes too.  A row per lane, straight from registers, would
// cost the load-store unit 32 lines per instruction.  bf16 matrices whose rows are
// no multiples of 16 bytes move through the same boxes, a row per step of the warp.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "activation.cuh"
#include "dropout.cuh"
#include "gemm_pair.cuh"
#include "launch.cuh"
#include "linear.h"
#include "prof.h"
#include "vec8.cuh"

namespace fbob {
namespace lin {
namespace {

using namespace tc;

constexpr int kThreads = 352;
constexpr int kEpWarps = 8;
constexpr int kTmemCols = 512;
constexpr int kBufCols = 256;  // accumulator columns per tile in flight
constexpr int kSlots = 2;      // boxes in flight per input and warp

template <int LAYOUT, int EP, int BN_>
struct Cfg {
  static constexpr int BN = BN_;
  static constexpr bool A_MN = LAYOUT == kTN;
  static constexpr bool B_MN = LAYOUT != kNT;
  static constexpr int A_BYTES = 128 * kBK * 2;
  static constexpr int B_BYTES = BN / 2 * kBK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NIN = EP == kForward ? 1 : EP == kSecond ? 2 : 0;
  static constexpr int BOXES = 2 + NIN * kSlots;  // of a warp: two outgoing, then the incoming ones
  static constexpr int ROOM = 229376 - kEpWarps * BOXES * kBoxBytes;
  static constexpr int NST = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
  static constexpr int BOX_OFF = NST * STAGE;
  static constexpr int SMEM = BOX_OFF + kEpWarps * BOXES * kBoxBytes;
  static_assert(SMEM + 2048 <= 232448, "shared memory budget");
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// Byte offset of 16-byte chunk c of row r in a box (64-byte swizzle).
__device__ __forceinline__ uint32_t box_at(uint32_t r, uint32_t c) { return r * 64 + ((c ^ ((r >> 1) & 3u)) << 4); }
// ... of element e of row r.
__device__ __forceinline__ uint32_t box_element(uint32_t r, uint32_t e) { return box_at(r, e >> 3) + (e & 7u) * 2; }

__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// 32 bf16 (HALF: fp16) values of this lane's row out of a box.
template <bool HALF>
__device__ __forceinline__ void read_box(uint32_t box, float* v) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (uint32_t c = 0; c < 4; ++c) {
    const uint4 u = ld_shared_v4(box + box_at(lane, c));
    if constexpr (HALF) {
      half8(u, v + 8 * c);
      continue;
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * c + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * c + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// A warp's 32 rows x 32 columns of an fp32 matrix at (y, x), a row per lane;
// `whole`: rows start on 32 bytes.
__device__ __forceinline__ void read_rows(const float* p, long long ld, bool live, int y, int x, int N, float* v) {
  const float* o = p + (size_t)(live ? y : 0) * ld + x;
  const bool vec = (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 4 == 0;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    if (vec && live && x + j + 4 <= N) {
      const float4 f = *reinterpret_cast<const float4*>(o + j);
      v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j + q] = live && x + j + q < N ? o[j + q] : 0.f;
    }
  }
}
__device__ __forceinline__ void write_rows(float* p, long long ld, bool live, int y, int x, int N, const float* v) {
  if (!live) return;
  float* o = p + (size_t)y * ld + x;
  const bool whole = (reinterpret_cast<uintptr_t>(p) & 31) == 0 && ld % 8 == 0;
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    if (whole && x + j + 8 <= N) {
      st_global_v8(o + j, reinterpret_cast<const uint32_t*>(v + j));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (x + j + q < N) o[j + q] = v[j + q];
      }
    }
  }
}

// 32 values of a vector at x, the same in all lanes (0 beyond N, or without one).
template <bool FP32>
__device__ __forceinline__ float column(const void* p, int x, int N) {
  const int n = x + (int)(threadIdx.x & 31);
  if (!p || n >= N) return 0.f;
  return FP32 ? static_cast<const float*>(p)[n] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[n]);
}

struct Ep {
  const GemmArgs& p;
  Outbox out;
  const Dropper& drop;
  int rows, N;

  // bf16 results leave through the map, or from the box row by row.
  __device__ __forceinline__ void put(const CUtensorMap* map, void* base, bool mapped, int x, int y,
                                      const uint32_t (&w)[16]) {
    if (mapped) {
      if (y < rows && x < N) out.put(map, x, y, w);
      return;
    }
    const uint32_t lane = threadIdx.x & 31, box = out.smem;
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // planes may be leaving from here
    __syncwarp();
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) st_shared_v4(box + box_at(lane, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    uint16_t* o = static_cast<uint16_t*>(base) + (size_t)y * p.ep.in_ld + x + lane;
    const bool in = x + (int)lane < N;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      if (in && y + r < rows) o[(size_t)r * p.ep.in_ld] = ld_shared_u16(box + box_element(r, lane));
    }
  }

  // HALF: in fp16, as z is kept beside bf16 tensors.
  template <bool FP32, bool HALF = false>
  __device__ __forceinline__ void result(const CUtensorMap* map, void* base, int x, int y, const float* v) {
    if constexpr (FP32) {
      const int row = y + (int)(threadIdx.x & 31);
      write_rows(static_cast<float*>(base), p.ep.in_ld, row < rows, row, x, N, v);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = HALF ? half_pair(v[2 * j], v[2 * j + 1]) : pack_bf16x2(v[2 * j], v[2 * j + 1]);
      put(map, base, p.ep.out_map, x, y, w);
    }
  }

  // As bf16 planes: plane k holds the rounding of what planes 0..k-1 left.
  __device__ __forceinline__ void planes(const CUtensorMap* maps, int n, int x, int y, float* v) {
    for (int k = 0; k < n; ++k) {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        const float2 f = __bfloat1622float2(h);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
        // an infinite value has no remainder (inf - inf would make one)
        v[2 * j] = isinf(f.x) ? 0.f : v[2 * j] - f.x;
        v[2 * j + 1] = isinf(f.y) ? 0.f : v[2 * j + 1] - f.y;
      }
      if (y < rows && x < N) out.put(maps + k, x, y, w);
    }
  }
};

// The incoming boxes of a warp: box `slot` of input i; bar[slot] counts the bytes of
// all inputs' boxes of a slot.
struct Inbox {
  uint32_t smem;
  uint64_t* bar;
  const GemmArgs* p;
  int n;         // inputs that are there
  bool mapped;
  int issued, taken;  // slots filled and read so far

  __device__ __forceinline__ const CUtensorMap* map(int i) const { return &p->in[p->ep.in0 ? i : i + 1]; }
  __device__ __forceinline__ const uint16_t* base(int i) const {
    return static_cast<const uint16_t*>(p->ep.in0 && i == 0 ? p->ep.in0 : p->ep.in1);
  }
  __device__ __forceinline__ uint32_t box(int slot, int i) const { return smem + (slot * n + i) * kBoxBytes; }

  // Start the loads of the warp's next box, at column x and row y.
  __device__ __forceinline__ void fetch(int x, int y) {
    if (n == 0) return;
    const int slot = issued % kSlots;
    ++issued;
    if (mapped) {
      if ((threadIdx.x & 31) == 0) {
        mbar_arrive_expect_tx(&bar[slot], n * kBoxBytes);
        for (int i = 0; i < n; ++i) tma_load_2d(box(slot, i), map(i), smem_u32(&bar[slot]), x, y);
      }
      return;
    }
    const int lane = threadIdx.x & 31;
    const bool in = x + lane < p->N;
    for (int i = 0; i < n; ++i) {
      const uint16_t* q = base(i) + (size_t)y * p->ep.in_ld + x + lane;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 16) {
        uint16_t v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = in && y + r0 + r < p->M ? q[(size_t)(r0 + r) * p->ep.in_ld] : (uint16_t)0;
#pragma unroll
        for (int r = 0; r < 16; ++r) st_shared_u16(box(slot, i) + box_element(r0 + r, lane), v[r]);
      }
    }
    __syncwarp();
  }
  // The oldest box has arrived (its slot), or -1 when the block gives up.
  __device__ __forceinline__ int wait(const Waiter& w) {
    const int slot = taken % kSlots;
    if (n && mapped && !__all_sync(0xffffffffu, mbar_wait(&bar[slot], (taken / kSlots) & 1, w))) return -1;
    return slot;
  }
  __device__ __forceinline__ void release() {
    __syncwarp();  // all lanes have read the box
    ++taken;
  }
  // Nothing may be in flight towards a block that has ended.
  __device__ __forceinline__ void drain() {
    if (!mapped) return;
    for (; taken < issued; ++taken) mbar_wait_drain(&bar[taken % kSlots], (taken / kSlots) & 1, kDrainNs);
  }
};

// 32 columns (from x) of a tile for this thread's row y0 + lane; in0, in1: the
// values of the inputs there.
template <int EP, bool FP32>
__device__ __forceinline__ void finish(Ep& e, float* v, float bias, const float* in0, float* in1, int x, int y0,
                                       int split) {
  const EpArgs& a = e.p.ep;
  const int lane = threadIdx.x & 31, row = y0 + lane;
  if constexpr (EP == kForward || EP == kSecond) {
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
    }
  }
  if constexpr (EP == kForward) {
    if (a.out1) e.result<FP32, true>(e.p.out + 1, a.out1, x, y0, v);
    act_values<FP32, 32>(a.act, v);
    if (e.drop.on) {
#pragma unroll
      for (int g = 0; g < 4; ++g) e.drop.apply8((uint32_t)(x >> 3) + g, (uint32_t)row, v + 8 * g);
    }
    if (a.in0) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] += in0[j];
    }
    e.result<FP32>(e.p.out, a.out0, x, y0, v);
  } else if constexpr (EP == kSecond) {
    // v = t; in0 = z, in1 = dy
    const bool live = row < e.rows;
    float a1[32], a2[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) a1[j] = in0[j];
    act_slopes<FP32, true, 32>(a.act, a1, a2);
    if (e.drop.on) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float m[8];
        e.drop.factors8((uint32_t)(x >> 3) + g, (uint32_t)row, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // what is dropped is 0 whatever stands there
          const int c = 8 * g + j;
          const bool kept = m[j] != 0.f;
          v[c] = kept ? v[c] : 0.f;
          in1[c] = kept ? in1[c] * m[j] : 0.f;
          a1[c] = kept ? a1[c] : 0.f;
          a2[c] = kept ? a2[c] : 0.f;
        }
      }
    }
    const float scale = e.drop.on ? e.drop.scale : 1.f;
    if (a.out0) {
      float g[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) g[j] = scale * v[j] * a1[j];
      e.result<FP32>(e.p.out, a.out0, x, y0, g);
    }
    if (a.dz_planes) {
#pragma unroll
      for (int j = 0; j < 32; ++j) a1[j] *= in1[j];
      e.planes(e.p.out + 2 + kPlanes, a.dz_planes, x, y0, a1);
    }
    if (a.q_planes || a.sums) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = live ? v[j] * in1[j] * a2[j] : 0.f;
      if (a.q_planes) {
        float q[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) q[j] = v[j];
        e.planes(e.p.out + 2, a.q_planes, x, y0, q);
      }
      if (a.sums) {
        // lane c ends with the sum over the lanes of their v[c]: halves of the
        // columns change sides, 16 values, 8, ...
#pragma unroll
        for (int h = 16; h > 0; h >>= 1) {
          const bool up = lane & h;
#pragma unroll
          for (int j = 0; j < h; ++j) {
            const float give = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, give, h);
          }
        }
        if (y0 < e.rows && x + lane < e.N) a.sums[(size_t)(y0 / 32) * a.ld + x + lane] = v[0];
      }
    }
  } else if constexpr (EP == kSlab) {
    float* o = a.slab + ((size_t)split * e.rows + row) * a.ld + x;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {  // ld is a multiple of 8
      if (row < e.rows && x + j < a.ld) st_global_v8(o + j, reinterpret_cast<const uint32_t*>(v + j));
    }
  } else {
    e.result<FP32>(e.p.out, a.out0, x, y0, v);
  }
}

template <int LAYOUT, int EP, bool FP32, bool HELD, int BN>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ GemmArgs p) {
  using C = Cfg<LAYOUT, EP, BN>;
  constexpr int H = BN / 2, CHUNKS = H / 32;  // columns of an epilogue thread
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Ctrl ctrl;
  __shared__ uint64_t in_bar[kEpWarps][kSlots];
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
    for (int w = 0; w < kEpWarps; ++w) {
      for (int s = 0; s < kSlots; ++s) mbar_init(&in_bar[w][s], 1);
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
  const Tiles ts{(p.M + kTileM - 1) / kTileM, (p.N + BN - 1) / BN, p.splits, (p.K + kBK - 1) / kBK};
  const int total = ts.count(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int chain_steps = p.chain;
  auto chain_end = [chain_steps](int kc, int k1) { return HELD ? min(kc + chain_steps, k1) : k1; };

  if (warp == 8 || warp == 10) {
    // ------------------------------------------- TMA: warp 8 loads A, warp 10 loads B
    const bool is_a = warp == 8;
    if (live) {  // the whole warp runs the loop; one lane issues (elect.sync)
      const uint32_t full0 = map_rank(smem_u32(&ctrl.full[0]), 0);
      Place<C::NST> at;
      long long issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        int m, n;
        ts.at(t, m, n);
        const int split = ts.split(t);
        const int row = m * kTileM + (int)rank * 128, col = n * BN + (int)rank * (BN / 2);
        const int k0 = ts.k_first(split), k1 = ts.k_first(split + 1);
        for (int kc = k0; ok && kc < k1; kc = chain_end(kc, k1)) {
          const int ke = chain_end(kc, k1);
          for (int s = 0; ok && s < p.nseg; ++s) {
            const CUtensorMap* ma = &p.a[p.seg[s].a];
            const CUtensorMap* mb = &p.b[p.seg[s].b];
            for (int k = kc; k < ke; ++k, ++issued, at.next()) {
              const int st = at.s;
              if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.empty[st], at.pass ^ 1, wt)))) break;
              if (p.stall && issued == 0) continue;  // test hook: nothing fills the first stage
              const uint32_t bar = full0 + 8 * st;
              const uint32_t da = sm0 + st * C::STAGE, db = da + C::A_BYTES;
              if (is_a) {
                if (rank == 0) mbar_expect_tx_w(&ctrl.full[st], 2 * C::STAGE);
                if (C::A_MN) {
                  tma_load_2d_pair(da, ma, bar, row, k * kBK);
                  tma_load_2d_pair(da + 8192, ma, bar, row + 64, k * kBK);
                } else {
                  tma_load_2d_pair(da, ma, bar, k * kBK, row);
                }
              } else if (C::B_MN) {
                tma_load_2d_pair(db, mb, bar, col, k * kBK);
                if (BN == 256) tma_load_2d_pair(db + 8192, mb, bar, col + 64, k * kBK);
              } else {
                tma_load_2d_pair(db, mb, bar, k * kBK, col);
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
      constexpr uint32_t id = idesc_bf16(kTileM, BN, C::A_MN, C::B_MN);
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
          for (int s = 0; ok && s < p.nseg; ++s) {
            for (int k = kc; k < ke; ++k, at.next()) {
              const int st = at.s;
              ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.full[st], at.pass, wt));
              if (!ok) break;
              tc_fence_after();
              const uint32_t more = s > 0 || k > kc;  // the accumulator holds a product already
              const uint32_t a = desc_lo(sm0 + st * C::STAGE, lbo_a);
              const uint32_t b = desc_lo(sm0 + st * C::STAGE + C::A_BYTES, lbo_b);
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk)
                mma_ss_pair(d, a + kk * step_a, b + kk * step_b, id, kk > 0 ? 1u : more);
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
    const int half = warp >> 2, quarter = (warp & 3) * 32;
    const uint32_t lane = (uint32_t)quarter << 16;
    const uint32_t freed = map_rank(smem_u32(&ctrl.tile_empty[0]), 0);
    const uint32_t boxes = sm0 + C::BOX_OFF + warp * C::BOXES * kBoxBytes;
    const Dropper drop(p.ep.drop);
    Ep e{p, Outbox{boxes, 0}, drop, p.M, p.N};
    Inbox in{boxes + 2 * kBoxBytes, in_bar[warp], &p, 0, p.ep.in_map != 0, 0, 0};
    if (C::NIN > 0 && !FP32) in.n = (p.ep.in0 != nullptr) + (C::NIN > 1 && p.ep.in1 != nullptr);
    // the warp's boxes in order: chunk c of its tiles
    auto fetch = [&](int t, int c) {
      if (C::NIN == 0 || in.n == 0) return;
      if (c >= CHUNKS) c -= CHUNKS, t += pairs;
      if (t >= total) return;
      int m, n;
      ts.at(t, m, n);
      in.fetch(n * BN + half * H + 32 * c, m * kTileM + (int)rank * 128 + quarter);
    };
    int chain = 0;
    bool ok = live;
    if (ok) {
#pragma unroll
      for (int c = 0; c < kSlots; ++c) fetch(pair, c);
    }
    for (int t = pair; ok && t < total; t += pairs) {
      int m, n;
      ts.at(t, m, n);
      const int split = ts.split(t);
      const int y0 = m * kTileM + (int)rank * 128 + quarter, x0 = n * BN + half * H;
      float sum[HELD ? H : 1];
      int buf = 0;
      if constexpr (HELD) {
#pragma unroll
        for (int j = 0; j < H; ++j) sum[j] = 0.f;
        const int k0 = ts.k_first(split), k1 = ts.k_first(split + 1);
        for (int kc = k0; kc < k1; kc = chain_end(kc, k1), ++chain) {
          buf = chain & 1;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.tile_full[buf], (chain >> 1) & 1, wt)))) break;
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < CHUNKS; ++q) {
            float v[32];
            tmem_ld32(tb + lane + buf * kBufCols + half * H + q * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[q * 32 + j] += v[j];
          }
          tc_fence_before();
          __syncwarp();
          if ((tid & 31) == 0) mbar_arrive_relaxed(freed + buf * 8);
        }
      } else {
        buf = chain & 1;
        // warp-uniform: the TMEM loads that follow are warp-collective
        ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.tile_full[buf], (chain >> 1) & 1, wt));
        tc_fence_after();
        ++chain;
      }
      if (!ok) break;
      const Acc<HELD> acc{tb + lane + buf * kBufCols + half * H, sum, freed + buf * 8};
#pragma unroll(HELD ? CHUNKS : 1)
      for (int c = 0; c < CHUNKS; ++c) {
        float v[32], in0[32], in1[32];
        const int x = x0 + 32 * c;
        const float bias = EP == kForward || EP == kSecond ? column<FP32>(p.ep.bias, x, p.N) : 0.f;
        acc.load(32 * c, 32 * c, v);
        if (c + 1 == CHUNKS) acc.done();
        if constexpr (C::NIN > 0) {
          if constexpr (FP32) {
            const int row = y0 + (tid & 31);
            if (p.ep.in0) read_rows(static_cast<const float*>(p.ep.in0), p.ep.in_ld, row < p.M, row, x, p.N, in0);
            if (C::NIN > 1 && p.ep.in1)
              read_rows(static_cast<const float*>(p.ep.in1), p.ep.in_ld, row < p.M, row, x, p.N, in1);
          } else if (in.n) {
            const int slot = in.wait(wt);
            if (!(ok = slot >= 0)) break;
            if (p.ep.in0) read_box<EP == kSecond>(in.box(slot, 0), in0);
            if (C::NIN > 1 && p.ep.in1) read_box<false>(in.box(slot, p.ep.in0 ? 1 : 0), in1);
            in.release();
            fetch(t, c + kSlots);
          }
          if (!p.ep.in0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) in0[j] = 0.f;
          }
          if (C::NIN > 1 && !p.ep.in1) {
#pragma unroll
            for (int j = 0; j < 32; ++j) in1[j] = 0.f;
          }
        }
        __syncwarp();
        finish<EP, FP32>(e, v, bias, in0, in1, x, y0, split);
      }
    }
    in.drain();
    e.out.drain();
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

template <int LAYOUT, int EP, bool FP32, bool HELD, int BN>
cudaError_t launch_as(const GemmArgs& g, const char* name, cudaStream_t s) {
  using C = Cfg<LAYOUT, EP, BN>;
  auto kernel = linear_kernel<LAYOUT, EP, FP32, HELD, BN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((g.M + kTileM - 1) / kTileM) * ((g.N + BN - 1) / BN) * g.splits;
  if (tiles == 0) return cudaSuccess;
  const long long pairs = sm_count() / 2;
  prof_begin(s, name);
  e = chained(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kThreads), C::SMEM, 2, s, g);
  prof_end(s);
  return e;
}

// Sums over slabs have tiles of 256 columns only (their number fills the device);
// the second order's of 128 where chains are held: its epilogue needs the registers.
template <int LAYOUT, int EP, bool FP32, bool HELD>
cudaError_t launch_tile(int tile_n, const GemmArgs& g, const char* name, cudaStream_t s) {
  if constexpr (!(EP == kSecond && HELD)) {
    if (tile_n == 256 || EP == kSlab) return launch_as<LAYOUT, EP, FP32, HELD, 256>(g, name, s);
  }
  if constexpr (EP != kSlab) return launch_as<LAYOUT, EP, FP32, HELD, 128>(g, name, s);
}

template <int LAYOUT, int EP>
cudaError_t launch(int tile_n, const GemmArgs& g, const char* name, cudaStream_t s) {
  if (g.fp32) return launch_tile<LAYOUT, EP, true, true>(tile_n, g, name, s);
  if (g.chain) return launch_tile<LAYOUT, EP, false, true>(tile_n, g, name, s);
  return launch_tile<LAYOUT, EP, false, false>(tile_n, g, name, s);
}

}  // namespace
}  // namespace lin
}  // namespace fbob
