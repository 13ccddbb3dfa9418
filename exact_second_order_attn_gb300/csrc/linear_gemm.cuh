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
// Roles of a block's warps: the first eight or sixteen epilogue (thread = accumulator
// row, the warpgroups take equal parts of the columns), then the TMA producer of A, MMA
// issue (the leader block's) with TMEM allocation, and the producer of B.  Sixteen where
// the epilogue computes (forward, second order): with eight, two per scheduler, it
// waited for its own results (30 % issue; gelu_tanh, 8192 x 2048 from 768 columns 44 us,
// its second order 90 us).  Barriers: full[s] of the
// leader counts both blocks' bytes; empty[s] and tile_full[b] are signalled in both
// blocks by the MMAs' commit; tile_empty[b] of the leader counts the epilogue warps of
// the pair.  Every wait is bounded.  Blocks are persistent: pair i takes
// tiles i, i + pairs, ...
//
// What the epilogue reads beside the accumulator (the residual; z and dy of the
// second order) comes in boxes of a warp's 32 rows x 32 columns: bulk tensor loads
// ahead of their use, which run under the products of the tile that the warp waits
// for; results leave in such boxes too (y from its residual's, q and dz from z's and
// dy's).  A row per lane, straight from registers,
// would cost the load-store unit 32 lines per instruction.  bf16 matrices whose rows
// are no multiples of 16 bytes move through the same boxes, a row per step of the
// warp.  The elementwise work goes by eight columns, 16 bytes of each box and one
// call of dropout's generator, so that little of it is live at a time.
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

constexpr int kTmemCols = 512;
constexpr int kBufCols = 256;   // accumulator columns per tile in flight
constexpr int kMaxStages = 8;   // of the barriers in Ctrl
constexpr int kRoom = 229376;   // bytes of stages and boxes

template <int EP>
constexpr bool kIsSecond = EP == kSecond || EP == kSecondTerms;

template <int LAYOUT, int EP, bool HELD, int BN_>
struct Cfg {
  static constexpr int BN = BN_;
  static constexpr bool A_MN = LAYOUT == kTN;
  static constexpr bool B_MN = LAYOUT != kNT;
  static constexpr int A_BYTES = 128 * kBK * 2;
  static constexpr int B_BYTES = BN / 2 * kBK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NIN = EP == kForward ? 1 : kIsSecond<EP> ? 2 : 0;
  static constexpr int WARPS = !HELD && (EP == kForward || EP == kSecond) ? 16 : 8;  // of the epilogue
  static constexpr int THREADS = 32 * (WARPS + 3);
  static constexpr int H = BN / (WARPS / 4);  // columns of an epilogue thread
  static_assert(kRoom + 2048 <= 232448, "shared memory budget");
  // Boxes of a warp: kForward y, z; kSecond z, dy, gdy; else two outgoing ones, then the inputs'.
  static int boxes(const GemmArgs& g) {
    return EP == kForward ? 1 + (g.ep.out1 != nullptr) : EP == kSecond ? 3 : EP == kSlab ? 0 : 2 + NIN;
  }
  static int stages(const GemmArgs& g) {
    const int n = (kRoom - WARPS * boxes(g) * kBoxBytes) / STAGE;
    return n < kMaxStages ? n : kMaxStages;
  }
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

// A place in the ring of stages and its pass over the ring.
struct Ring {
  int n, s = 0;
  uint32_t pass = 0;
  __device__ __forceinline__ void next() {
    if (++s == n) s = 0, pass ^= 1;
  }
};

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
    copy_rows(box, base, x, y);
  }
  // A box that has been written (and synchronised) goes out row by row.
  __device__ __forceinline__ void copy_rows(uint32_t box, void* base, int x, int y) {
    const uint32_t lane = threadIdx.x & 31;
    uint16_t* o = static_cast<uint16_t*>(base) + (size_t)y * p.ep.in_ld + x + lane;
    const bool in = x + (int)lane < N;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      if (in && y + r < rows) o[(size_t)r * p.ep.in_ld] = ld_shared_u16(box + box_element(r, lane));
    }
  }
  // The boxes of a chunk leave: `to` is their place by bulk store (null map: by rows).
  __device__ __forceinline__ void leave(uint32_t box, const CUtensorMap* map, int x, int y) {
    if ((threadIdx.x & 31) == 0 && y < rows && x < N)
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(box), "r"(x), "r"(y)
                   : "memory");
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
      for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      if (k + 1 < n) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          // an infinite value has no remainder (inf - inf would make one)
          const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
          v[2 * j] = isinf(lo) ? 0.f : v[2 * j] - lo;
          v[2 * j + 1] = isinf(hi) ? 0.f : v[2 * j + 1] - hi;
        }
      }
      if (y < rows && x < N) out.put(maps + k, x, y, w);
    }
  }
};

// The incoming boxes of a warp, one for each input; the barrier counts their bytes.
struct Inbox {
  uint32_t smem;
  uint64_t* bar;
  const GemmArgs* p;
  int n;  // inputs that are there
  bool mapped;
  int issued, taken;  // chunks asked for and used so far

  __device__ __forceinline__ const CUtensorMap* map(int i) const { return &p->in[p->ep.in0 ? i : i + 1]; }
  __device__ __forceinline__ const uint16_t* base(int i) const {
    return static_cast<const uint16_t*>(p->ep.in0 && i == 0 ? p->ep.in0 : p->ep.in1);
  }
  __device__ __forceinline__ uint32_t box(int i) const { return smem + i * kBoxBytes; }

  // Start the loads of the warp's next chunk, at column x and row y.  The boxes are
  // free: nothing reads them any more, bulk stores included.
  __device__ __forceinline__ void fetch(int x, int y) {
    ++issued;
    if (mapped) {
      if ((threadIdx.x & 31) == 0) {
        mbar_arrive_expect_tx(bar, n * kBoxBytes);
        for (int i = 0; i < n; ++i) tma_load_2d(box(i), map(i), smem_u32(bar), x, y);
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
        for (int r = 0; r < 16; ++r) st_shared_u16(box(i) + box_element(r0 + r, lane), v[r]);
      }
    }
    __syncwarp();
  }
  // The chunk's boxes have arrived; false when the block gives up.
  __device__ __forceinline__ bool wait(const Waiter& w) {
    const bool ok = n == 0 || !mapped || __all_sync(0xffffffffu, mbar_wait(bar, taken & 1, w));
    if (ok) ++taken;
    return ok;
  }
  // Nothing may be in flight towards a block that has ended.
  __device__ __forceinline__ void drain() {
    if (mapped && n && taken < issued) mbar_wait_drain(bar, taken & 1, kDrainNs);
  }
};

__device__ __forceinline__ void commit_stores() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The warp's boxes have been read: by its stores, and by its lanes.
__device__ __forceinline__ void boxes_free() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

__device__ __forceinline__ void box_values(uint32_t box, int g, float* v) {
  const uint4 u = ld_shared_v4(box + box_at(threadIdx.x & 31, g));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void box_store(uint32_t box, int g, const float* v) {
  const uint4 u = bf16x8(v);
  st_shared_v4(box + box_at(threadIdx.x & 31, g), u.x, u.y, u.z, u.w);
}

// 8 consecutive fp32 columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Lane 4 c of the warp returns the sum over the lanes of their v[c], c < 8.
__device__ __forceinline__ float sum_columns8(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 16; h > 2; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int j = 0; j < h / 4; ++j) {
      const float give = up ? v[j] : v[j + h / 4], keep = up ? v[j + h / 4] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// Lane c of the warp returns the sum over the lanes of their v[c]: halves of the
// columns change sides, 16 values, 8, ...
__device__ __forceinline__ float sum_columns(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 16; h > 0; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int j = 0; j < h; ++j) {
      const float give = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  return v[0];
}

// t[j] += bias of the columns 8 g + j, out of the warp's 32 in shared memory.
__device__ __forceinline__ void add_bias(const float* bias, int g, float* t) {
  const float4 a = *reinterpret_cast<const float4*>(bias + 8 * g), b = *reinterpret_cast<const float4*>(bias + 8 * g + 4);
  t[0] += a.x, t[1] += a.y, t[2] += a.z, t[3] += a.w, t[4] += b.x, t[5] += b.y, t[6] += b.z, t[7] += b.w;
}

// bf16 tensors, 32 columns (from x) of the forward for the row y0 + lane: y into the
// box `out`, where its residual is, z into the one behind.
template <int ACT>
__device__ __forceinline__ void forward_values(Ep& e, float* v, const float* bias, uint32_t out, int x, int y0) {
  const EpArgs& a = e.p.ep;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float* w = v + 8 * g;
    if (a.bias) add_bias(bias, g, w);
    if (ACT != kActNone && a.out1)
      st_shared_v4(out + kBoxBytes + box_at(lane, g), half_pair(w[0], w[1]), half_pair(w[2], w[3]),
                   half_pair(w[4], w[5]), half_pair(w[6], w[7]));
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = act_value<ACT, false>(w[j]);
    if (e.drop.on) e.drop.apply8((uint32_t)(x >> 3) + g, (uint32_t)(y0 + lane), w);
    if (a.in0) {
      float r[8];
      box_values(out, g, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] += r[j];
    }
    box_store(out, g, w);
  }
}
__device__ __forceinline__ void forward_bf16(Ep& e, float* v, const float* bias, uint32_t out, int x, int y0) {
  const EpArgs& a = e.p.ep;
  switch (a.act) {
    case kActRelu: forward_values<kActRelu>(e, v, bias, out, x, y0); break;
    case kActGelu: forward_values<kActGelu>(e, v, bias, out, x, y0); break;
    case kActGeluTanh: forward_values<kActGeluTanh>(e, v, bias, out, x, y0); break;
    case kActSilu: forward_values<kActSilu>(e, v, bias, out, x, y0); break;
    default: forward_values<kActNone>(e, v, bias, out, x, y0);
  }
  if (a.out_map) fence_proxy_async_smem();
  __syncwarp();
  if (a.out_map) {
    e.leave(out, e.p.out, x, y0);
    if (a.out1) e.leave(out + kBoxBytes, e.p.out + 1, x, y0);
    commit_stores();
  } else {
    e.copy_rows(out, a.out0, x, y0);
    if (a.out1) e.copy_rows(out + kBoxBytes, a.out1, x, y0);
  }
}

// bf16 tensors with one term of dz and q, the second order: v = t; the boxes of z and
// dy (those that are there), over which q and dz are written, and gdy's.  Eight
// columns at a time come out of the accumulator: 104 registers a thread hold no more.
template <int ACT, bool HELD>
__device__ __forceinline__ void second_values(Ep& e, const Acc<HELD>& acc, int c, bool last, const float* bias,
                                              uint32_t zbox, uint32_t dybox, uint32_t out, int x, int y0) {
  const EpArgs& a = e.p.ep;
  const int lane = threadIdx.x & 31;
  const bool live = y0 + lane < e.rows;
#pragma unroll(HELD ? 4 : 1)
  for (int g = 0; g < 4; ++g) {
    float t[8];
    if constexpr (HELD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = acc.sum[c + 8 * g + j];
    } else {
      __syncwarp();
      tmem_ld8(acc.tmem + c + 8 * g, t);
      if (last && g == 3) acc.done();
    }
    if (a.bias) add_bias(bias, g, t);
    float a1[8], a2[8], dy[8], m[8];
    if (ACT != kActNone) half8(ld_shared_v4(zbox + box_at(lane, g)), a1);
#pragma unroll
    for (int j = 0; j < 8; ++j) a1[j] = act_slope<ACT, false, true>(a1[j], a2[j]);
    if (a.in1) box_values(dybox, g, dy);
    if (e.drop.on) {
      e.drop.factors8((uint32_t)(x >> 3) + g, (uint32_t)(y0 + lane), m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // what is dropped is 0 whatever stands there
        const bool kept = m[j] != 0.f;
        t[j] = kept ? t[j] : 0.f;
        a1[j] = kept ? a1[j] * e.drop.scale : 0.f;
        a2[j] = kept ? a2[j] * e.drop.scale : 0.f;
        if (a.in1) dy[j] = kept ? dy[j] : 0.f;
      }
    }
    if (a.out0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = t[j] * a1[j];
      box_store(out, g, m);
    }
    if (a.dz_planes) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a1[j] *= dy[j];
      box_store(dybox, g, a1);
    }
    if (a.q_planes || a.sums) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = live ? t[j] * dy[j] * a2[j] : 0.f;
      if (a.q_planes) box_store(zbox, g, t);
      if (a.sums) {
        const float s = sum_columns8(t);
        const int n = x + 8 * g + lane / 4;
        if (lane % 4 == 0 && y0 < e.rows && n < e.N) a.sums[(size_t)(y0 / 32) * a.ld + n] = s;
      }
    }
  }
}
template <bool HELD>
__device__ __forceinline__ void second_bf16(Ep& e, const Acc<HELD>& v, int c, bool last, const float* bias,
                                            uint32_t zbox, uint32_t dybox, uint32_t out, int x, int y0) {
  const EpArgs& a = e.p.ep;
  switch (a.act) {
    case kActRelu: second_values<kActRelu>(e, v, c, last, bias, zbox, dybox, out, x, y0); break;
    case kActGelu: second_values<kActGelu>(e, v, c, last, bias, zbox, dybox, out, x, y0); break;
    case kActGeluTanh: second_values<kActGeluTanh>(e, v, c, last, bias, zbox, dybox, out, x, y0); break;
    case kActSilu: second_values<kActSilu>(e, v, c, last, bias, zbox, dybox, out, x, y0); break;
    default: second_values<kActNone>(e, v, c, last, bias, zbox, dybox, out, x, y0);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (a.out0 && a.out_map) e.leave(out, e.p.out, x, y0);
  if (a.dz_planes) e.leave(dybox, e.p.out + 2 + kPlanes, x, y0);
  if (a.q_planes) e.leave(zbox, e.p.out + 2, x, y0);
  commit_stores();
  if (a.out0 && !a.out_map) e.copy_rows(out, a.out0, x, y0);
}

// 32 columns (from x) of a tile for this thread's row y0 + lane, fp32 tensors, two
// terms of dz and q, or no more than a result; in0, in1: the values of the inputs.
template <int EP, bool FP32>
__device__ __forceinline__ void finish(Ep& e, float* v, float bias, const float* in0, float* in1, int x, int y0,
                                       int split) {
  const EpArgs& a = e.p.ep;
  const int lane = threadIdx.x & 31, row = y0 + lane;
  if constexpr (EP == kForward || kIsSecond<EP>) {
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
  } else if constexpr (EP == kSecondTerms) {
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
        const float total = sum_columns(v);
        if (y0 < e.rows && x + lane < e.N) a.sums[(size_t)(y0 / 32) * a.ld + x + lane] = total;
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
__global__ void __launch_bounds__(Cfg<LAYOUT, EP, HELD, BN>::THREADS, 1)
    linear_kernel(const __grid_constant__ GemmArgs p) {
  using C = Cfg<LAYOUT, EP, HELD, BN>;
  constexpr int H = C::H, CHUNKS = H / 32, EW = C::WARPS;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Ctrl ctrl;
  __shared__ uint64_t in_bar[EW];
  __shared__ __align__(16) float bias_row[EW][32];
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  allow_next();

  if (tid == 0) {
    ctrl.abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&ctrl.full[s], 1);
      mbar_init(&ctrl.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl.tile_full[b], 1);
      mbar_init(&ctrl.tile_empty[b], 2 * EW);
    }
    for (int w = 0; w < EW; ++w) mbar_init(&in_bar[w], 1);
    mbar_init(&ctrl.drain, 1);
    fence_mbar_init();
    if ((smem_u32(smem) & 1023u) != 0u) {
      ctrl.abort_flag = 1;
      atomicOr(p.err, kErrTimeout);
    }
  }
  if (warp == EW + 1) {
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

  const int nst = p.stages;
  if (warp == EW || warp == EW + 2) {
    // ------------------------------------------- TMA: one warp loads A, the other B
    const bool is_a = warp == EW;
    if (live) {  // the whole warp runs the loop; one lane issues (elect.sync)
      const uint32_t full0 = map_rank(smem_u32(&ctrl.full[0]), 0);
      Ring at{nst};
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
      for (long long i = issued > nst ? issued - nst : 0; i < issued; ++i) {
        const int st = (int)(i % nst);
        if (rank == 0 && !ok) mbar_wait_drain(&ctrl.full[st], (i / nst) & 1, kDrainNs);
        if (ok) ok = mbar_wait(&ctrl.empty[st], (i / nst) & 1, wt);
      }
      if (!ok && rank != 0) {  // this block's loads count on the leader's barriers: give them time to land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kDrainNs) {
        }
      }
    }
  } else if (warp == EW + 1) {
    // ------------------------------------------------------------------ MMA
    if (live && rank == 0) {
      constexpr uint32_t id = idesc_bf16(kTileM, BN, C::A_MN, C::B_MN);
      constexpr uint32_t lbo_a = C::A_MN ? 8192 : 16, lbo_b = C::B_MN ? 8192 : 16;
      constexpr uint32_t step_a = C::A_MN ? 2048 >> 4 : 32 >> 4, step_b = C::B_MN ? 2048 >> 4 : 32 >> 4;
      Ring at{nst};
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
    const int part = warp >> 2, quarter = (warp & 3) * 32;
    const uint32_t lane = (uint32_t)quarter << 16;
    const uint32_t freed = map_rank(smem_u32(&ctrl.tile_empty[0]), 0);
    const uint32_t boxes = sm0 + nst * C::STAGE + warp * p.boxes * kBoxBytes;
    const Dropper drop(p.ep.drop);
    Ep e{p, Outbox{boxes, 0}, drop, p.M, p.N};
    Inbox in{EP == kSecondTerms ? boxes + 2 * kBoxBytes : boxes, &in_bar[warp], &p, 0, p.ep.in_map != 0, 0, 0};
    if (C::NIN > 0 && !FP32) in.n = (p.ep.in0 != nullptr) + (C::NIN > 1 && p.ep.in1 != nullptr);
    // chunk c of the warp's tiles, counted from tile t
    auto fetch = [&](int t, int c) {
      if (C::NIN == 0 || in.n == 0) return;
      if (c >= CHUNKS) c -= CHUNKS, t += pairs;
      if (t >= total) return;
      int m, n;
      ts.at(t, m, n);
      in.fetch(n * BN + part * H + 32 * c, m * kTileM + (int)rank * 128 + quarter);
    };
    int chain = 0;
    bool ok = live;
    if (ok) fetch(pair, 0);
    for (int t = pair; ok && t < total; t += pairs) {
      int m, n;
      ts.at(t, m, n);
      const int split = ts.split(t);
      const int y0 = m * kTileM + (int)rank * 128 + quarter, x0 = n * BN + part * H;
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
            tmem_ld32(tb + lane + buf * kBufCols + part * H + q * 32, v);
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
      const Acc<HELD> acc{tb + lane + buf * kBufCols + part * H, sum, freed + buf * 8};
#pragma unroll(HELD ? CHUNKS : 1)
      for (int c = 0; c < CHUNKS; ++c) {
        float v[32];
        const int x = x0 + 32 * c;
        const float bias = EP == kForward || kIsSecond<EP> ? column<FP32>(p.ep.bias, x, p.N) : 0.f;
        if constexpr (C::NIN > 0 && !FP32) {
          if (!(ok = in.wait(wt))) break;
        }
        if constexpr (EP != kSecond) {
          acc.load(32 * c, 32 * c, v);
          if (c + 1 == CHUNKS) acc.done();
        }
        if constexpr (!FP32 && (EP == kForward || EP == kSecond)) {
          if (p.ep.bias) {
            bias_row[warp][tid & 31] = bias;
            __syncwarp();
          }
          if (EP == kForward)
            forward_bf16(e, v, bias_row[warp], boxes, x, y0);
          else
            second_bf16(e, acc, 32 * c, c + 1 == CHUNKS, bias_row[warp], in.box(0), in.box(p.ep.in0 ? 1 : 0), boxes + 2 * kBoxBytes, x, y0);
          boxes_free();
          fetch(t, c + 1);
        } else if constexpr (EP == kSecondTerms && !FP32) {
          float in0[32], in1[32];
          if (p.ep.in0) read_box<true>(in.box(0), in0);
          if (p.ep.in1) read_box<false>(in.box(p.ep.in0 ? 1 : 0), in1);
          __syncwarp();
          fetch(t, c + 1);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (!p.ep.in0) in0[j] = 0.f;
            if (!p.ep.in1) in1[j] = 0.f;
          }
          finish<EP, FP32>(e, v, bias, in0, in1, x, y0, split);
        } else {
          float in0[32], in1[32];
          const int row = y0 + (tid & 31);
          if (C::NIN > 0 && p.ep.in0)
            read_rows(static_cast<const float*>(p.ep.in0), p.ep.in_ld, row < p.M, row, x, p.N, in0);
          if (C::NIN > 1 && p.ep.in1)
            read_rows(static_cast<const float*>(p.ep.in1), p.ep.in_ld, row < p.M, row, x, p.N, in1);
          if (C::NIN > 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!p.ep.in0) in0[j] = 0.f;
              if (C::NIN > 1 && !p.ep.in1) in1[j] = 0.f;
            }
          }
          __syncwarp();
          finish<EP, FP32>(e, v, bias, in0, in1, x, y0, split);
        }
      }
    }
    in.drain();
    e.out.drain();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither block ends, or frees tensor memory, before the other is done
  if (warp == EW + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tb, kTmemCols);
  }
}

template <int LAYOUT, int EP, bool FP32, bool HELD, int BN>
cudaError_t launch_as(GemmArgs g, const char* name, cudaStream_t s) {
  using C = Cfg<LAYOUT, EP, HELD, BN>;
  auto kernel = linear_kernel<LAYOUT, EP, FP32, HELD, BN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)((g.M + kTileM - 1) / kTileM) * ((g.N + BN - 1) / BN) * g.splits;
  if (tiles == 0) return cudaSuccess;
  const long long pairs = sm_count() / 2;
  g.boxes = C::boxes(g), g.stages = C::stages(g);
  prof_begin(s, name);
  e = chained(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(C::THREADS), kRoom, 2, s, g);
  prof_end(s);
  return e;
}

// Sums over slabs have tiles of 256 columns only (their number fills the device);
// forward and second order of 128 where their epilogues need the registers.
template <int LAYOUT, int EP, bool FP32, bool HELD>
cudaError_t launch_tile(int tile_n, const GemmArgs& g, const char* name, cudaStream_t s) {
  if constexpr (!(EP == kSecondTerms || ((EP == kSecond || EP == kForward) && HELD))) {
    if (tile_n == 256 || EP == kSlab) return launch_as<LAYOUT, EP, FP32, HELD, 256>(g, name, s);
  }
  if constexpr (EP != kSlab) return launch_as<LAYOUT, EP, FP32, HELD, 128>(g, name, s);
}

template <int LAYOUT, int EP>
cudaError_t launch(int tile_n, const GemmArgs& g, const char* name, cudaStream_t s) {
  if constexpr (EP != kSecond) {
    if (g.fp32) return launch_tile<LAYOUT, EP, true, true>(tile_n, g, name, s);
  }
  if (g.chain) return launch_tile<LAYOUT, EP, false, true>(tile_n, g, name, s);
  return launch_tile<LAYOUT, EP, false, false>(tile_n, g, name, s);
}

}  // namespace
}  // namespace lin
}  // namespace fbob
