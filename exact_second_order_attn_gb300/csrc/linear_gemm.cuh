// The matrix products of linear layers on the fifth generation tensor cores, with
// the layer's elementwise work in the epilogue.
//
// One or two problems in a launch (dx and dW read the same dz and share their waves:
// 768 -> 2304, 8192 tokens, 52 us in two launches, 39 in one).  C[256 x BN] = sum over
// segments of A_seg B_seg^T per pair of thread blocks (cta_group::2): each block holds
// its 128 rows of A and its half of B's rows of every 64-column stage; the
// accumulator's 128 rows x BN columns lie in the block's tensor memory, two of them, so
// the epilogue of one tile runs under the products of the next.
//
// fp32 operands are three bf16 terms each, and the six products of terms that reach
// 2^-16 of the first are summed, smallest first, out of one stage that holds all terms
// (a stage for each product would load twice the bytes, at 12 TB/s what bound it).  The
// tensor cores drop the bits of a step's sum below the accumulator's last one, so there
// a chain ends after 64 columns and the epilogue threads add the chains up in
// registers (HELD); so do sums of bf16 operands over more than 16,384 terms, every
// 16,384 (3e-5 of the result).
//
// Roles of a block's warps: the first eight, twelve or sixteen epilogue (thread =
// accumulator row, the warpgroups take equal parts of the columns), then the TMA
// producer of A, MMA issue (the leader block's) with TMEM allocation, and the producer
// of B.  Sixteen (twelve for 192 columns) where the epilogue computes: with eight, two
// per scheduler, it waited for its own results (30 % issue; gelu_tanh, 8192 x 2048 from
// 768 columns 44 us, its second order 90 us; 26 and 70 now).  Barriers: full[s] of the
// leader counts both blocks' bytes; empty[s] and tile_full[b] are signalled in both
// blocks by the MMAs' commit; tile_empty[b] of the leader counts the epilogue warps of
// the pair.  Every wait is bounded.  Blocks are persistent: pair i takes tiles i, i +
// pairs, ...
//
// What the epilogue reads beside the accumulator (the residual; z and dy of the second
// order) comes in boxes of a warp's 32 rows x 32 columns: bulk tensor loads ahead of
// their use, which run under the products of the tile that the warp waits for; results
// leave in such boxes too (y from its residual's, q and dz from z's and dy's).  A row
// per lane, straight from registers, would cost the load-store unit 32 lines per
// instruction.  bf16 matrices whose rows are no multiples of 16 bytes move through the
// same boxes, a row per step of the warp.  The elementwise work goes by eight columns,
// 16 bytes of each box and one call of dropout's generator, in a loop that is not
// unrolled: with all 32 columns in line the code did not fit the instruction cache
// (fp32 gelu forward, 1021 x 2048 from 512 columns, 49 us; 33 in the loop).
//
// Measured on 8192 tokens, bf16, alone: 768 -> 2304 forward 22.5 us (1,290 TFLOP/s), dx
// and dW 37 (1,570); 4096 -> 11,008 under the power cap 440 (1,680) and 795 (1,860).
// Bound by the loads of the stages (a tile of K = 768 takes 4.1 us where its MMAs need
// 3.2) and, in short launches, by their ends: 1.2 us until the first stage, 2.9 for the
// last tile's epilogue, 2 until the next kernel's start.
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

template <int LAYOUT, int EP, bool FP32, bool HELD, int BN_>
struct Cfg {
  static constexpr int BN = BN_;
  static constexpr bool B_MN = LAYOUT == kGradients;
  static constexpr int A_BYTES = 128 * kBK * 2;
  static constexpr int B_BYTES = BN / 2 * kBK * 2;
  // fp32: a stage holds all terms of both operands for the six products
  static constexpr bool TERMS = FP32;
  static constexpr int STAGE = (A_BYTES + B_BYTES) * (TERMS ? kPlanes : 1);  // [A.. | B..]
  static constexpr int B_OFF = A_BYTES * (TERMS ? kPlanes : 1);
  static constexpr int NIN = EP == kForward ? 1 : kIsSecond<EP> ? 2 : 0;
  // of the epilogue; 64 columns a thread of tiles of 256 and 192
  static constexpr int WARPS = EP == kForward || EP == kSecond ? (BN == 192 ? 12 : 16) : 8;
  static constexpr int THREADS = 32 * (WARPS + 3);
  static constexpr int H = BN / (WARPS / 4);  // columns of an epilogue thread
  static_assert(kRoom + 2048 <= 232448, "shared memory budget");
  // Boxes of a warp: of y and its residual, and z; of z and q, dy and dz, gdy, then the
  // further terms of q and dz in turn (fp32: of one's terms); of two results.
  static int boxes(const GemmArgs& g) {
    if (EP == kForward) return FP32 ? 0 : 1 + (g.ep.out1 != nullptr);
    return EP == kSecond ? 3 : EP == kSecondTerms ? (FP32 ? 3 : 5) : EP == kGradient && !FP32 ? 2 : 0;
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
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

// Eight columns from x of row y of an fp32 matrix [rows][N]; `live`: the row exists.
__device__ __forceinline__ bool whole8(const void* p, long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 31) == 0 && ld % 8 == 0;
}
__device__ __forceinline__ void read8(const float* p, long long ld, bool live, int y, int x, int N, float* v) {
  const float* o = p + (size_t)(live ? y : 0) * ld + x;
  if (live && whole8(p, ld) && x + 8 <= N) {
    load8<float, true>(o, 8, v);
  } else {
    load8<float, false>(o, live ? N - x : 0, v);
  }
}
__device__ __forceinline__ void write8(float* p, long long ld, bool live, int y, int x, int N, const float* v) {
  if (!live) return;
  float* o = p + (size_t)y * ld + x;
  if (whole8(p, ld) && x + 8 <= N) {
    st_global_v8(o, reinterpret_cast<const uint32_t*>(v));
  } else {
    store8<float, false>(o, N - x, v);
  }
}

// Lane j has column x + j of a vector (0 beyond N, or without one).
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
  int rows, N;      // of the tile's problem,
  long long ld;     // and its outputs' rows

  // bf16 results leave through the map, or from the box row by row.
  __device__ __forceinline__ void put(const CUtensorMap* map, void* base, bool mapped, int x, int y,
                                      const uint32_t (&w)[16]) {
    if (mapped) {
      if (y < rows && x < N) out.put(map, x, y, w);
      return;
    }
    const uint32_t lane = threadIdx.x & 31, box = out.smem;
    // (results of a launch's other problem may be leaving from here)
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) st_shared_v4(box + box_at(lane, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    copy_rows(box, base, x, y);
  }
  // A box that has been written (and synchronised) goes out row by row.
  __device__ __forceinline__ void copy_rows(uint32_t box, void* base, int x, int y) {
    const uint32_t lane = threadIdx.x & 31;
    uint16_t* o = static_cast<uint16_t*>(base) + (size_t)y * ld + x + lane;
    const bool in = x + (int)lane < N;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      if (in && y + r < rows) o[(size_t)r * ld] = ld_shared_u16(box + box_element(r, lane));
    }
  }
  // A box that has been written (and synchronised) leaves as a bulk tensor store.
  __device__ __forceinline__ void leave(uint32_t box, const CUtensorMap* map, int x, int y) {
    if ((threadIdx.x & 31) == 0 && y < rows && x < N)
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(box), "r"(x), "r"(y)
                   : "memory");
  }

  template <bool FP32>
  __device__ __forceinline__ void result(const Problem& q, int x, int y, const float* v) {
    if constexpr (FP32) {
      const int row = y + (int)(threadIdx.x & 31);
#pragma unroll
      for (int j = 0; j < 32; j += 8)
        write8(static_cast<float*>(q.out0), ld, row < rows, row, x + j, N, v + j);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      put(&q.out, q.out0, q.out_map, x, y, w);
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

  __device__ __forceinline__ const void* base(int i) const { return i == 0 ? p->ep.in0 : p->ep.in1; }
  __device__ __forceinline__ uint32_t box(int i) const { return smem + i * kBoxBytes; }

  // Start the loads of the warp's next chunk, at column x and row y.  The boxes are
  // free: nothing reads them any more, bulk stores included.
  __device__ __forceinline__ void fetch(int x, int y) {
    ++issued;
    if (mapped) {
      if ((threadIdx.x & 31) == 0) {
        mbar_arrive_expect_tx(bar, n * kBoxBytes);
        for (int i = 0; i < 2; ++i) {
          if (base(i)) tma_load_2d(box(i), p->in + i, smem_u32(bar), x, y);
        }
      }
      return;
    }
    const int lane = threadIdx.x & 31;
    const bool in = x + lane < p->prob[0].N;
    for (int i = 0; i < 2; ++i) {
      if (!base(i)) continue;
      const uint16_t* q = static_cast<const uint16_t*>(base(i)) + (size_t)y * p->ep.in_ld + x + lane;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 16) {
        uint16_t v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = in && y + r0 + r < p->prob[0].M ? q[(size_t)(r0 + r) * p->ep.in_ld] : (uint16_t)0;
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

// t[j] += bias of the columns 8 g + j, out of the warp's 32 in shared memory.
__device__ __forceinline__ void add_bias(const float* bias, int g, float* t) {
  const float4 a = *reinterpret_cast<const float4*>(bias + 8 * g), b = *reinterpret_cast<const float4*>(bias + 8 * g + 4);
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  add8(t, v);
}

// Where the elementwise epilogues find 32 columns of the product, eight at a time
// (more live values would not fit 104 registers, more code not the instruction cache):
// in the accumulator, which is handed back behind the last of them, or (HELD) where
// the sum of its chains has been put.
template <bool HELD>
struct Columns {
  uint32_t tmem, freed;
  bool last;
  __device__ __forceinline__ void load(int g, float* t) const {
    __syncwarp();  // the load is warp-collective
    tmem_ld8(tmem + 8 * g, t);
    if (!HELD && last && g == 3) Acc<false>{0, nullptr, freed}.done();
  }
};

// 32 columns (from x) of the forward for the row y0 + lane.  bf16: y into the box
// `out`, where its residual is, z into the one behind.
template <int ACT, bool FP32, bool HELD>
__device__ __forceinline__ void forward_values(Ep& e, const Columns<HELD>& in, const float* bias, uint32_t out, int x,
                                               int y0) {
  const EpArgs& a = e.p.ep;
  const int lane = threadIdx.x & 31, row = y0 + lane;
  const bool live = row < e.rows;
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    float v[8];
    in.load(g, v);
    if (a.bias) add_bias(bias, g, v);
    if (ACT != kActNone && a.out1) {
      if (FP32)
        write8(static_cast<float*>(a.out1), a.in_ld, live, row, x + 8 * g, e.N, v);
      else {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = ACT == kActRelu ? kept_sign(v[j]) : v[j];
        st_shared_v4(out + kBoxBytes + box_at(lane, g), half_pair(z[0], z[1]), half_pair(z[2], z[3]),
                     half_pair(z[4], z[5]), half_pair(z[6], z[7]));
      }
    }
    act_values8<ACT, FP32>(v);
    if (e.drop.on) e.drop.apply8((uint32_t)(x >> 3) + g, (uint32_t)row, v);
    if (a.in0) {
      float r[8];
      if (FP32)
        read8(static_cast<const float*>(a.in0), a.in_ld, live, row, x + 8 * g, e.N, r);
      else
        box_values(out, g, r);
      add8(v, r);
    }
    if (FP32)
      write8(static_cast<float*>(a.out0), a.in_ld, live, row, x + 8 * g, e.N, v);
    else
      box_store(out, g, v);
  }
}
template <bool FP32, bool HELD>
__device__ __forceinline__ void forward_chunk(Ep& e, const Columns<HELD>& in, const float* bias, uint32_t out, int x,
                                              int y0) {
  const EpArgs& a = e.p.ep;
  switch (a.act) {
    case kActRelu: forward_values<kActRelu, FP32>(e, in, bias, out, x, y0); break;
    case kActGelu: forward_values<kActGelu, FP32>(e, in, bias, out, x, y0); break;
    case kActGeluTanh: forward_values<kActGeluTanh, FP32>(e, in, bias, out, x, y0); break;
    case kActSilu: forward_values<kActSilu, FP32>(e, in, bias, out, x, y0); break;
    default: forward_values<kActNone, FP32>(e, in, bias, out, x, y0);
  }
  if (FP32) return;
  // before the box's bulk store, or its next bulk load, where y itself goes out row by row
  if (a.in_map || a.out_map) fence_proxy_async_smem();
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

// The box of term k of q (which = 0) or dz (1); fp32's terms of both take turns in three.
template <bool FP32>
__device__ __forceinline__ uint32_t term_box(uint32_t boxes, int which, int k) {
  return boxes + (FP32 ? k : k == 0 ? which : 1 + 2 * k + which) * kBoxBytes;
}
// v as n bf16 terms (one without TERMS): each holds the rounding of what the ones
// before it left.
template <bool FP32, bool TERMS>
__device__ __forceinline__ void store_terms(uint32_t boxes, int which, int n, int g, float* v) {
  box_store(term_box<FP32>(boxes, which, 0), g, v);
  if constexpr (TERMS) {
    for (int k = 1; k < n; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // an infinite value has no remainder (inf - inf would make one)
        const float h = __bfloat162float(__float2bfloat16_rn(v[j]));
        v[j] = isinf(h) ? 0.f : v[j] - h;
      }
      box_store(term_box<FP32>(boxes, which, k), g, v);
    }
  }
}

// 32 columns (from x) of the second order for the row y0 + lane: the product is t.
// bf16: z and dy are in the first two boxes, over which q and dz are written (PART is
// kAll).  fp32: z and dy come from memory, eight columns ahead; first what t makes, then
// (kDz) dz, in the boxes that q has left.
enum Part { kAll, kFromT, kDz };
template <int ACT, bool FP32, bool TERMS, bool HELD, int PART>
__device__ __forceinline__ void second_values(Ep& e, const Columns<HELD>& in, const float* bias, uint32_t boxes, int x,
                                              int y0) {
  const EpArgs& a = e.p.ep;
  const int lane = threadIdx.x & 31, row = y0 + lane;
  const bool live = row < e.rows;
  float z_next[8], dy_next[8];
  auto ahead = [&](int g) {
    if (ACT != kActNone) read8(static_cast<const float*>(a.in0), a.in_ld, live, row, x + 8 * g, e.N, z_next);
    if (a.in1) read8(static_cast<const float*>(a.in1), a.in_ld, live, row, x + 8 * g, e.N, dy_next);
  };
  if (FP32) ahead(0);
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    float t[8], a1[8], a2[8], dy[8], m[8];
    if (FP32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a1[j] = z_next[j], dy[j] = dy_next[j];
      if (g < 3) ahead(g + 1);
    } else {
      if (ACT != kActNone) half8(ld_shared_v4(boxes + box_at(lane, g)), a1);
      if (a.in1) box_values(boxes + kBoxBytes, g, dy);
    }
    if (PART != kDz) {
      in.load(g, t);
      if (a.bias && live) add_bias(bias, g, t);  // (rows past the last are 0)
    }
    act_slopes8<ACT, FP32, PART != kDz>(a1, a2);
    if (e.drop.on) {
      e.drop.factors8((uint32_t)(x >> 3) + g, (uint32_t)row, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // what is dropped is 0 whatever stands there
        const bool kept = m[j] != 0.f;
        a1[j] = kept ? a1[j] * e.drop.scale : 0.f;
        if (a.in1) dy[j] = kept ? dy[j] : 0.f;
        if (PART != kDz) {
          t[j] = kept ? t[j] : 0.f;
          a2[j] = kept ? a2[j] * e.drop.scale : 0.f;
        }
      }
    }
    if (PART != kDz && a.out0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = t[j];
      mul8(m, a1);
      if (FP32)
        write8(static_cast<float*>(a.out0), a.in_ld, live, row, x + 8 * g, e.N, m);
      else
        box_store(boxes + 2 * kBoxBytes, g, m);
    }
    if (PART != kFromT && a.dz_planes) {
      mul8(a1, dy);
      store_terms<FP32, TERMS>(boxes, 1, a.dz_planes, g, a1);
    }
    if (PART != kDz && (a.q_planes || a.sums)) {
      mul8(t, dy);
      mul8(t, a2);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = t[j];
      if (a.q_planes) store_terms<FP32, TERMS>(boxes, 0, a.q_planes, g, m);
      if (a.sums) {
        if (y0 + 32 > e.rows) {  // rows past the last: their t is 0 times uW, which need not be finite
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] = live ? t[j] : 0.f;
        }
        const float s = sum_columns8(t);
        const int n = x + 8 * g + lane / 4;
        if (lane % 4 == 0 && y0 < e.rows && n < e.N) a.sums[(size_t)(y0 / 32) * a.ld + n] = s;
      }
    }
  }
}
template <bool FP32, bool TERMS, int PART, bool HELD>
__device__ __forceinline__ void second_part(Ep& e, const Columns<HELD>& in, const float* bias, uint32_t boxes, int x,
                                            int y0) {
  switch (e.p.ep.act) {
    case kActRelu: second_values<kActRelu, FP32, TERMS, HELD, PART>(e, in, bias, boxes, x, y0); break;
    case kActGelu: second_values<kActGelu, FP32, TERMS, HELD, PART>(e, in, bias, boxes, x, y0); break;
    case kActGeluTanh: second_values<kActGeluTanh, FP32, TERMS, HELD, PART>(e, in, bias, boxes, x, y0); break;
    case kActSilu: second_values<kActSilu, FP32, TERMS, HELD, PART>(e, in, bias, boxes, x, y0); break;
    default: second_values<kActNone, FP32, TERMS, HELD, PART>(e, in, bias, boxes, x, y0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}
template <bool FP32, bool TERMS, bool HELD>
__device__ __forceinline__ void second_chunk(Ep& e, const Columns<HELD>& in, const float* bias, uint32_t boxes, int x,
                                             int y0) {
  const EpArgs& a = e.p.ep;
  second_part<FP32, TERMS, FP32 ? kFromT : kAll>(e, in, bias, boxes, x, y0);
  if (!FP32 && a.out0 && a.out_map) e.leave(boxes + 2 * kBoxBytes, e.p.out, x, y0);
  for (int k = 0; k < (TERMS ? a.q_planes : a.q_planes != 0); ++k)
    e.leave(term_box<FP32>(boxes, 0, k), e.p.out + 2 + k, x, y0);
  if (FP32 && a.dz_planes) {
    commit_stores();
    boxes_free();
    second_part<FP32, TERMS, kDz>(e, in, bias, boxes, x, y0);
  }
  for (int k = 0; k < (TERMS ? a.dz_planes : a.dz_planes != 0); ++k)
    e.leave(term_box<FP32>(boxes, 1, k), e.p.out + 2 + kPlanes + k, x, y0);
  commit_stores();
  if (!FP32 && a.out0 && !a.out_map) e.copy_rows(boxes + 2 * kBoxBytes, a.out0, x, y0);
}

// 32 columns (from x) of a gradient or a slab, for the row y0 + lane.
template <int EP, bool FP32>
__device__ __forceinline__ void finish(Ep& e, const Problem& q, const float* v, int x, int y0, int split) {
  if (EP == kSlab || q.slab) {
    const int row = y0 + (int)(threadIdx.x & 31);
    float* o = q.slab + ((size_t)split * e.rows + row) * q.slab_ld + x;
#pragma unroll
    for (int j = 0; j < 32; j += 8) {  // slab_ld is a multiple of 8
      if (row < e.rows && x + j < q.slab_ld) st_global_v8(o + j, reinterpret_cast<const uint32_t*>(v + j));
    }
  } else {
    e.result<FP32>(q, x, y0, v);
  }
}

// The tiles of a launch: those of the first problem, then those of the second.
struct Plan {
  Tiles first, second;
  int n0, total;
  __device__ __forceinline__ Plan(const GemmArgs& p, int bn)
      : first(tiles(p.prob[0], bn)), second(tiles(p.prob[1], bn)), n0(first.count()),
        total(n0 + (p.problems > 1 ? second.count() : 0)) {}
  static __device__ __forceinline__ Tiles tiles(const Problem& q, int bn) {
    return Tiles{(q.M + kTileM - 1) / kTileM, (q.N + bn - 1) / bn, q.splits, (q.K + kBK - 1) / kBK};
  }
};
// Where a tile lies and the steps of its contraction.
struct Place {
  int which, m, n, split, k0, k1, chain;
  __device__ __forceinline__ Place(const GemmArgs& p, const Plan& plan, int t) {
    which = t >= plan.n0;
    const Tiles& ts = which ? plan.second : plan.first;
    if (which) t -= plan.n0;
    ts.at(t, m, n);
    split = ts.split(t);
    k0 = ts.k_first(split), k1 = ts.k_first(split + 1);
    chain = p.prob[which].chain;
  }
  // the step at which a chain of the tensor cores that starts at kc ends
  template <bool HELD>
  __device__ __forceinline__ int end(int kc) const {
    return HELD && chain ? min(kc + chain, k1) : k1;
  }
};

template <int LAYOUT, int EP, bool FP32, bool HELD, int BN>
__global__ void __launch_bounds__(Cfg<LAYOUT, EP, FP32, HELD, BN>::THREADS, 1)
    linear_kernel(const __grid_constant__ GemmArgs p) {
  using C = Cfg<LAYOUT, EP, FP32, HELD, BN>;
  constexpr int H = C::H, CHUNKS = H / 32, EW = C::WARPS;
  constexpr bool ELEMENTWISE = EP == kForward || kIsSecond<EP>;
  static_assert(!(HELD && ELEMENTWISE) || BN == 128, "chains' sums lie behind the accumulators of 128 columns");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Ctrl ctrl;
  __shared__ uint64_t in_bar[EW];
  __shared__ __align__(16) float bias_row[EW][32];
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  allow_next();

  if (tid < 32) {  // a barrier or two per lane
    static_assert(kMaxStages == 8 && EW <= 32, "lanes below");
    if (tid < p.stages) mbar_init(&ctrl.full[tid], 1);
    if (tid >= 8 && tid - 8 < p.stages) mbar_init(&ctrl.empty[tid - 8], 1);
    if (tid == 16 || tid == 17) mbar_init(&ctrl.tile_full[tid - 16], 1);
    if (tid == 18 || tid == 19) mbar_init(&ctrl.tile_empty[tid - 18], 2 * EW);
    if (tid == 20) mbar_init(&ctrl.drain, 1);
    if (tid < EW) mbar_init(&in_bar[tid], 1);
    fence_mbar_init();
  }
  // The maps' descriptors are on their way while the kernel before this one ends.
  if (warp == EW || warp == EW + 2) {
    const int lane = tid & 31, seg = C::TERMS ? lane / kPlanes : lane, term = C::TERMS ? lane % kPlanes : 0;
    for (int i = 0; i < p.problems; ++i) {
      const Problem& q = p.prob[i];
      if (seg < q.nseg) prefetch_map(warp == EW ? &q.a[q.seg[seg].a + term] : &q.b[q.seg[seg].b + term]);
      if (EP == kGradient && warp == EW && lane == 31 && q.out_map && !q.slab) prefetch_map(&q.out);
    }
  } else if (ELEMENTWISE && warp == 1) {
    const EpArgs& e = p.ep;
    const int lane = tid & 31, k = lane % 4;
    if (lane < 2 && e.in_map && (lane ? e.in1 : e.in0)) prefetch_map(&p.in[lane]);
    if (lane >= 2 && lane < 4 && e.out_map && (k == 2 ? e.out0 : e.out1)) prefetch_map(&p.out[k - 2]);
    if (lane >= 4 && lane < 8 && k < e.q_planes) prefetch_map(&p.out[2 + k]);
    if (lane >= 8 && lane < 12 && k < e.dz_planes) prefetch_map(&p.out[2 + kPlanes + k]);
  }
  if (tid == 0) {
    ctrl.abort_flag = 0;
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
  const Plan plan(p, BN);
  const int total = plan.total, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
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
        const Place at_tile(p, plan, t);
        const Problem& q = p.prob[at_tile.which];
        const int row = at_tile.m * kTileM + (int)rank * 128, col = at_tile.n * BN + (int)rank * (BN / 2);
        const bool a_mn = LAYOUT == kGradients && q.a_mn;
        for (int kc = at_tile.k0; ok && kc < at_tile.k1; kc = at_tile.template end<HELD>(kc)) {
          const int ke = at_tile.template end<HELD>(kc);
          for (int s = 0; ok && s < q.nseg; ++s) {
            const CUtensorMap* ma = &q.a[q.seg[s].a];
            const CUtensorMap* mb = &q.b[q.seg[s].b];
            for (int k = kc; k < ke; ++k, ++issued, at.next()) {
              const int st = at.s;
              if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.empty[st], at.pass ^ 1, wt)))) break;
              if (p.stall && issued == 0) continue;  // test hook: nothing fills the first stage
              const uint32_t bar = full0 + 8 * st;
              if (is_a && rank == 0) mbar_expect_tx_w(&ctrl.full[st], 2 * C::STAGE);
#pragma unroll
              for (int i = 0; i < (C::TERMS ? kPlanes : 1); ++i) {
                const uint32_t da = sm0 + st * C::STAGE + i * C::A_BYTES;
                const uint32_t db = sm0 + st * C::STAGE + C::B_OFF + i * C::B_BYTES;
                if (is_a) {
                  if (a_mn) {
                    tma_load_2d_pair(da, ma + i, bar, row, k * kBK);
                    tma_load_2d_pair(da + 8192, ma + i, bar, row + 64, k * kBK);
                  } else {
                    tma_load_2d_pair(da, ma + i, bar, k * kBK, row);
                  }
                } else if (C::B_MN) {
                  tma_load_2d_pair(db, mb + i, bar, col, k * kBK);
                  if (BN == 256) tma_load_2d_pair(db + 8192, mb + i, bar, col + 64, k * kBK);
                } else {
                  tma_load_2d_pair(db, mb + i, bar, k * kBK, col);
                }
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
      constexpr uint32_t lbo_b = C::B_MN ? 8192 : 16, step_b = C::B_MN ? 2048 >> 4 : 32 >> 4;
      Ring at{nst};
      int chain = 0;  // accumulator buffers handed to the epilogue so far
      bool ok = true;
      for (int t = pair; ok && t < total; t += pairs) {
        const Place tile(p, plan, t);
        const Problem& q = p.prob[tile.which];
        const bool a_mn = LAYOUT == kGradients && q.a_mn;
        const uint32_t id = a_mn ? idesc_bf16(kTileM, BN, true, C::B_MN) : idesc_bf16(kTileM, BN, false, C::B_MN);
        const uint32_t lbo_a = a_mn ? 8192 : 16, step_a = a_mn ? 2048 >> 4 : 32 >> 4;
        for (int kc = tile.k0; ok && kc < tile.k1; kc = tile.template end<HELD>(kc)) {
          const int ke = tile.template end<HELD>(kc);
          uint32_t d = 0;
          auto open = [&]() {  // the chain's accumulator is free
            ok = __all_sync(0xffffffffu, wait_cluster(&ctrl.tile_empty[chain & 1], ((chain >> 1) & 1) ^ 1, wt));
            tc_fence_after();
            d = tb + (chain & 1) * kBufCols;
          };
          if (!C::TERMS) open();
          for (int s = 0; ok && s < q.nseg; ++s) {
            if (C::TERMS) open();  // (a chain is one step of one segment)
            for (int k = kc; ok && k < ke; ++k, at.next()) {
              const int st = at.s;
              ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.full[st], at.pass, wt));
              if (!ok) break;
              tc_fence_after();
              const uint32_t more = (!C::TERMS && s > 0) || k > kc;  // the accumulator holds a product already
              const uint32_t a = desc_lo(sm0 + st * C::STAGE, lbo_a);
              const uint32_t b = desc_lo(sm0 + st * C::STAGE + C::B_OFF, lbo_b);
              if constexpr (C::TERMS) {
                // the products of terms that reach 2^-16 of the first, smallest first
#pragma unroll
                for (int order = kPlanes - 1; order >= 0; --order) {
#pragma unroll
                  for (int i = order; i >= 0; --i) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                      mma_ss_pair(d, a + i * (C::A_BYTES >> 4) + kk * step_a,
                                  b + (order - i) * (C::B_BYTES >> 4) + kk * step_b, id,
                                  kk > 0 || i < kPlanes - 1 ? 1u : more);
                  }
                }
              } else {
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                  mma_ss_pair(d, a + kk * step_a, b + kk * step_b, id, kk > 0 ? 1u : more);
              }
              mma_commit_pair(&ctrl.empty[st]);
            }
            if (C::TERMS) mma_commit_pair(&ctrl.tile_full[chain & 1]), ++chain;
          }
          if (!C::TERMS) mma_commit_pair(&ctrl.tile_full[chain & 1]), ++chain;
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
    Ep e{p, Outbox{boxes, 0}, drop, p.prob[0].M, p.prob[0].N, p.ep.in_ld};
    Inbox in{boxes, &in_bar[warp], &p, 0, p.ep.in_map != 0, 0, 0};
    if (C::NIN > 0 && !FP32) in.n = (p.ep.in0 != nullptr) + (C::NIN > 1 && p.ep.in1 != nullptr);
    // chunk c of the warp's tiles, counted from tile t
    auto fetch = [&](int t, int c) {
      if (C::NIN == 0 || in.n == 0) return;
      if (c >= CHUNKS) c -= CHUNKS, t += pairs;
      if (t >= total) return;
      const Place tile(p, plan, t);
      in.fetch(tile.n * BN + part * H + 32 * c, tile.m * kTileM + (int)rank * 128 + quarter);
    };
    int chain = 0;
    bool ok = live;
    if (ok && C::NIN > 0 && in.n) {
      // The first boxes are wanted when a whole tile's products are done: behind them the
      // first stages would come late (second order: products began 5 us late).
      __nanosleep(1000);
      fetch(pair, 0);
    }
    for (int t = pair; ok && t < total; t += pairs) {
      const Place tile(p, plan, t);
      const Problem& q = p.prob[tile.which];
      const int y0 = tile.m * kTileM + (int)rank * 128 + quarter, x0 = tile.n * BN + part * H;
      if (LAYOUT == kGradients) e.rows = q.M, e.N = q.N, e.ld = q.N;
      // (on its way while the tile's products are)
      float bias = ELEMENTWISE ? column<FP32>(p.ep.bias, x0, e.N) : 0.f;
      float sum[HELD ? H : 1];
      int buf = 0;
      if constexpr (HELD) {
#pragma unroll
        for (int j = 0; j < H; ++j) sum[j] = 0.f;
        int chains = 0;
        for (int kc = tile.k0; kc < tile.k1; kc = tile.template end<HELD>(kc)) chains += C::TERMS ? q.nseg : 1;
        for (int i = 0; i < chains; ++i, ++chain) {
          buf = chain & 1;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctrl.tile_full[buf], (chain >> 1) & 1, wt)))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            float v[32];
            tmem_ld32(tb + lane + buf * kBufCols + part * H + c * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c * 32 + j] += v[j];
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
      if constexpr (ELEMENTWISE) {
        uint32_t from = tb + lane + buf * kBufCols + part * H;
        if constexpr (HELD) {  // (columns 128.. of the first buffer)
          from = tb + lane + 128 + part * H;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < H; j += 16) tmem_st16_nowait(from + j, reinterpret_cast<const uint32_t*>(sum) + j);
          tmem_st_wait();
        }
        for (int c = 0; c < CHUNKS; ++c) {
          const int x = x0 + 32 * c;
          if (p.ep.bias) {
            bias_row[warp][tid & 31] = bias;
            __syncwarp();
            if (c + 1 < CHUNKS) bias = column<FP32>(p.ep.bias, x + 32, e.N);
          }
          if (!FP32 && !(ok = in.wait(wt))) break;
          const Columns<HELD> cols{from + 32 * c, freed + buf * 8, c + 1 == CHUNKS};
          if constexpr (EP == kForward)
            forward_chunk<FP32>(e, cols, bias_row[warp], boxes, x, y0);
          else
            second_chunk<FP32, EP == kSecondTerms>(e, cols, bias_row[warp], boxes, x, y0);
          boxes_free();
          if (!FP32) fetch(t, c + 1);
        }
      } else {
        const Acc<HELD> acc{tb + lane + buf * kBufCols + part * H, sum, freed + buf * 8};
#pragma unroll(HELD ? CHUNKS : 1)
        for (int c = 0; c < CHUNKS; ++c) {
          float v[32];
          acc.load(32 * c, 32 * c, v);
          if (c + 1 == CHUNKS) acc.done();
          __syncwarp();
          finish<EP, FP32>(e, q, v, x0 + 32 * c, y0, tile.split);
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
  using C = Cfg<LAYOUT, EP, FP32, HELD, BN>;
  auto kernel = linear_kernel<LAYOUT, EP, FP32, HELD, BN>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  if (e != cudaSuccess) return e;
  long long tiles = 0;
  for (int i = 0; i < g.problems; ++i) {
    const Problem& q = g.prob[i];
    tiles += (long long)((q.M + kTileM - 1) / kTileM) * ((q.N + BN - 1) / BN) * q.splits;
  }
  if (tiles == 0) return cudaSuccess;
  const long long pairs = sm_count() / 2;
  g.boxes = C::boxes(g), g.stages = C::stages(g);
  prof_begin(s, name);
  e = chained(kernel, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(C::THREADS), kRoom, 2, s, g);
  prof_end(s);
  return e;
}

// Gradients and slabs have tiles of 256 columns only (their number fills the device);
// forward and second order of 128 where chains are held, whose sums lie behind them.
template <int LAYOUT, int EP, bool FP32, bool HELD>
cudaError_t launch_tile(int tile_n, const GemmArgs& g, const char* name, cudaStream_t s) {
  constexpr bool GRADIENT = EP == kSlab || EP == kGradient;
  if constexpr (GRADIENT || !(EP == kSecondTerms || HELD)) {
    if (tile_n == 256) return launch_as<LAYOUT, EP, FP32, HELD, 256>(g, name, s);
  }
  if constexpr (!GRADIENT && !(EP == kSecondTerms || HELD)) {
    if (tile_n == 192) return launch_as<LAYOUT, EP, FP32, HELD, 192>(g, name, s);
  }
  if constexpr (!GRADIENT) {
    if (tile_n == 128) return launch_as<LAYOUT, EP, FP32, HELD, 128>(g, name, s);
  }
  return cudaErrorInvalidValue;
}

template <int LAYOUT, int EP>
cudaError_t launch(int tile_n, const GemmArgs& g, const char* name, cudaStream_t s) {
  if constexpr (EP != kSecond) {
    if (g.fp32) return launch_tile<LAYOUT, EP, true, true>(tile_n, g, name, s);
  }
  if (g.prob[0].chain || (g.problems > 1 && g.prob[1].chain)) return launch_tile<LAYOUT, EP, false, true>(tile_n, g, name, s);
  return launch_tile<LAYOUT, EP, false, false>(tile_n, g, name, s);
}

}  // namespace
}  // namespace lin
}  // namespace fbob
