// Parts of the persistent product kernels on block pairs (the linear head's
// cross entropy, linear layers): barriers of a block, the ring of stages, the
// order of the tiles, and the epilogue warps' way to accumulators and outputs.
#pragma once

#include "tc_pair.cuh"

namespace fbob {
namespace tc {

constexpr int kGroupM = 8;        // row tiles per raster group
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kBoxBytes = 32 * 32 * 2;  // a box: a warp's 32 rows x 32 columns of bf16

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

}  // namespace tc
}  // namespace fbob
