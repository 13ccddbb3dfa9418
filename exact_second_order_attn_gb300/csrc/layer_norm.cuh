// Layer norm over rows of D elements: what its three kernels share.
//
//   y = w xh + b,  xh = (x - m(x)) r,  r = (m((x - m(x))^2) + eps)^(-1/2)
//
// with m() the mean over the row.  The kernels are bound by memory, so a row
// is read once and kept in registers between its reductions, in its memory
// format; arithmetic is on fp32 pairs, since at one instruction per element
// and operation the issue slots would bind next.  A row belongs to a warp up
// to 1024 columns and to a whole thread block above that (up to 256 threads of
// 16 elements, 512 of 16, 512 of 32).  Owners take several rows at a time where
// the registers allow, which shares the reductions' latency.  Row statistics
// are fp32 and two-pass: the variance is summed over x - m(x), not over x^2.
//
// Rows arrive through a ring in shared memory, filled by untiled bulk copies
// several rows ahead of their owner, so the bytes in flight do not depend on
// registers or on where the owners stand in their reductions.
//
// Rows off 16-byte bounds (D not a multiple of 16 bytes, shifted tensors): a
// copy's bounds are moved outwards to the neighbouring rows' bytes, and a
// thread's vectors are cut at 16-byte addresses, not at columns.  Every block
// takes rows of one residue of the row index, so that all of them lie the same
// way: its vectors then hold the same columns in every row, and the weights are
// staged once, shifted, in shared memory.  Only vectors at a row's ends are
// handled element by element.
//
// Measured (bf16, copy rate 6.79 TB/s): 32,768 x 4096 forward 87 us, 6.2 TB/s,
// backward 137 us, 5.9 TB/s, at about half of the issue slots; 8192 x 768 7 and
// 12 us, of which the launch and the first loads are half.
#pragma once

#include <cuda_runtime.h>

#include "copy_bounds.h"
#include "internal.h"
#include "launch.cuh"
#include "prof.h"
#include "rowvec.cuh"
#include "tc_ptx.cuh"

namespace fbob {
namespace ln {

using row::all;
using row::bf16;
using row::F2;
using row::kUnits;
using row::mad;
using row::Raw;
using row::total;
using row::Unit;

constexpr int kWarps = 8;         // owners per block when a warp owns a row
constexpr int kWarpCols = 1024;   // widest row of one warp
constexpr int kMaxStages = 8;
constexpr uint64_t kDrainNs = 200000000ull;

// Who owns a row, and the most threads of the kernel's blocks.
enum Owner { kWarp, kBlock256, kBlock512 };
template <int OWN>
constexpr int kMaxThreads = OWN == kBlock512 ? 512 : 256;
// Weights are staged in shared memory where the rows lie off 16-byte bounds
// (blocks of 512 threads never take such rows as vectors) and read in place
// otherwise: staging costs a launch of few rows 4 us.
template <int VEC, bool EVEN>
constexpr bool kStaged = VEC > 1 && !EVEN;

// Rows taken at a time: N tensors' rows of E elements in at most 48 registers.
template <typename T, int E, int N>
constexpr int kRows = N * E * (int)sizeof(T) / 4 <= 8 ? 4 : N * E * (int)sizeof(T) / 4 <= 24 ? 2 : 1;

// Blocks per multiprocessor (of kMaxThreads; smaller ones fit more often), and
// their shared memory.
template <typename T, int E, int OWN>
constexpr int kResident = OWN == kBlock512 || E * (int)sizeof(T) > 64 ? 1 : 2;
constexpr int kRingMemory = 200 * 1024;
// The dynamic shared memory that every kernel is allowed.  The allowance belongs
// to the kernel, not to the launch, and host threads may launch one kernel for
// different sizes at once, so it is one number for all of them: a ring and staged
// weights take 200 KB at most, static arrays 4.1 KB of the 227 KB of a block.
constexpr int kDynamicMemory = 220 * 1024;
inline int blocks_per_max(int threads) { return threads < 256 ? 256 / threads : 1; }

// Where a block's rows lie against 16-byte bounds, and this thread's columns:
// vector i starts at column at(i), which may be below 0 or run past D where the
// row starts off a bound (shift elements after it).
template <int VEC, int E, int OWN, bool EVEN>
struct Cols {
  static constexpr int NV = E / VEC;
  int D, shift, lane, threads;
  __device__ __forceinline__ Cols(int D_, int shift_)
      : D(D_),
        shift(shift_),
        lane(OWN != kWarp ? threadIdx.x : threadIdx.x & 31),
        threads(OWN != kWarp ? blockDim.x : 32) {}
  __device__ __forceinline__ int at(int i) const { return (i * threads + lane) * VEC - (EVEN ? 0 : shift); }
  __device__ __forceinline__ bool any(int i) const { return at(i) < D; }
  __device__ __forceinline__ bool whole(int i) const { return VEC == 1 || EVEN || (at(i) >= 0 && at(i) + VEC <= D); }
  __device__ __forceinline__ bool has(int i, int j) const { return at(i) + j >= 0 && at(i) + j < D; }
};

// N tensors' rows on their way to one owner, R at a time.  Blocks take the
// rows of residue blockIdx.x % period; an owner's step holds the rows r,
// r + period, .. r + (R - 1) period, its next one starts `step` rows further on.
// EVEN: every row starts and ends on a 16-byte bound, and period is 1.
template <typename T, int N, int R, int VEC, int OWN, bool EVEN>
struct Ring {
  static constexpr int kOwners = OWN == kWarp ? kWarps : 1;
  struct Bars {
    uint64_t full[kOwners][kMaxStages];
  };

  const char* base[N];
  long long rows, first, step;
  int period, row_bytes, slot, stages, edge;
  uint32_t smem;    // this owner's slots: [stage][tensor][row]
  uint64_t* full;   // and barriers
  bool issuer;

  static __host__ __device__ int slot_bytes(int D) {
    return EVEN ? D * (int)sizeof(T) : (D * (int)sizeof(T) + 15) / 16 * 16 + 16;
  }

  __device__ __forceinline__ Ring(const T* const (&x)[N], long long n, int D, int P, int S, char* dyn, Bars& bars) {
    const int owner = OWN == kWarp ? threadIdx.x >> 5 : 0;
#pragma unroll
    for (int k = 0; k < N; ++k) base[k] = reinterpret_cast<const char*>(x[k]);
    rows = n, stages = S, row_bytes = D * (int)sizeof(T), slot = slot_bytes(D), period = EVEN ? 1 : P;
    edge = copy_edge(row_bytes);
    first = ((long long)(blockIdx.x / period) * kOwners + owner) * R * period + blockIdx.x % period;
    step = (long long)(gridDim.x / period) * kOwners * R * period;
    smem = tc::smem_u32(dyn) + owner * S * N * R * slot;
    full = bars.full[owner];
    issuer = (OWN == kWarp ? threadIdx.x & 31 : threadIdx.x) == 0;
    if (issuer) {
      for (int s = 0; s < S; ++s) tc::mbar_init(full + s, 1);
      tc::fence_mbar_init();
    }
    if (OWN == kWarp) __syncwarp();
    else __syncthreads();
    for (int k = 0; k < S; ++k) fill(k, first + k * step);
  }

  // Elements between a 16-byte bound and the start of this block's rows.
  __device__ __forceinline__ int shift() const {
    return EVEN ? 0
                : (int)((reinterpret_cast<uintptr_t>(base[0]) + (long long)(blockIdx.x % period) * row_bytes) & 15) /
                      (int)sizeof(T);
  }
  __device__ __forceinline__ bool live(long long r, int j) const { return r + j * period < rows; }

  __device__ __forceinline__ bool at_end(long long r) const { return copy_at_end(r, rows, edge); }
  // Bounds of the bytes that the copy for row r of tensor b brings.
  __device__ __forceinline__ void bounds(const char* b, long long r, uintptr_t& lo, uintptr_t& hi) const {
    copy_bounds(reinterpret_cast<uintptr_t>(b), rows, row_bytes, edge, r, lo, hi);
  }

  __device__ __forceinline__ void copy(uint32_t dst, uintptr_t src, uint32_t bytes, uint64_t* bar) const {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
  }

  // Start the copies of the owner's k-th step, whose first row is r.
  __device__ __forceinline__ void fill(int k, long long r) const {
    if (!issuer || r >= rows) return;
    const int s = k % stages;
    if constexpr (EVEN) {  // the step's rows are adjacent
      const uint32_t bytes = (uint32_t)min((long long)R, rows - r) * row_bytes;
      tc::mbar_arrive_expect_tx(full + s, N * bytes);
#pragma unroll
      for (int n = 0; n < N; ++n)
        copy(smem + (s * N + n) * R * slot, reinterpret_cast<uintptr_t>(base[n]) + r * row_bytes, bytes, full + s);
    } else {
      uint32_t bytes = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!live(r, j)) break;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          uintptr_t lo, hi;
          bounds(base[n], r + j * period, lo, hi);
          bytes += (uint32_t)(hi - lo);
        }
      }
      tc::mbar_arrive_expect_tx(full + s, bytes);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!live(r, j)) break;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          uintptr_t lo, hi;
          bounds(base[n], r + j * period, lo, hi);
          const uintptr_t at = reinterpret_cast<uintptr_t>(base[n]) + (r + j * period) * row_bytes;
          const uint32_t dst = smem + ((s * N + n) * R + j) * slot + (uint32_t)(lo - (at & ~(uintptr_t)15));
          if (hi > lo) copy(dst, lo, (uint32_t)(hi - lo), full + s);
        }
      }
    }
  }

  // Wait for the owner's k-th step (a limit bounds it; false: give up).
  __device__ __forceinline__ bool wait(int k, long long r, unsigned int* err, unsigned long long limit) const {
    uint64_t* bar = full + k % stages;
    const uint32_t parity = (k / stages) & 1;
    bool ok = tc::mbar_try_wait(bar, parity);
    if (!ok) {
      const uint64_t t0 = tc::globaltimer_ns();
      while (!(ok = tc::mbar_try_wait(bar, parity)) && tc::globaltimer_ns() - t0 <= limit) {
      }
    }
    if (!__all_sync(0xffffffffu, ok)) {
      if (!ok) atomicOr(err, kErrTimeout);
      if (issuer) {  // nothing may still be on its way to this block's memory when it ends
        for (int s = 0; s < stages && r + s * step < rows; ++s)
          tc::mbar_wait_drain(full + (k + s) % stages, ((k + s) / stages) & 1, kDrainNs);
      }
      return false;
    }
    return true;
  }

  // This thread's part of row j of the k-th step (first row r) of tensor n;
  // zero outside the row.
  template <int E>
  __device__ __forceinline__ void read(int k, long long r, int j, int n, Raw<T, VEC> (&v)[E / VEC],
                                       const Cols<VEC, E, OWN, EVEN>& c) const {
    const uint32_t at_slot = smem + (((k % stages) * N + n) * R + j) * slot;
    if constexpr (EVEN) {
      const T* in = static_cast<const T*>(__cvta_shared_to_generic(at_slot));
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
        v[i].clear();
        if (c.any(i) && live(r, j)) v[i].load(in + c.at(i));
      }
    } else {
      const long long mine_row = r + j * period;
      if (mine_row >= rows) {
#pragma unroll
        for (int i = 0; i < c.NV; ++i) v[i].clear();
        return;
      }
      const T* src = reinterpret_cast<const T*>(base[n] + mine_row * row_bytes);
      const uintptr_t at = reinterpret_cast<uintptr_t>(src);
      // column 0 in the slot; VEC == 1 takes rows of any residue
      const T* in = static_cast<const T*>(__cvta_shared_to_generic(at_slot)) +
                    (VEC == 1 ? (at & 15) / sizeof(T) : c.shift);
      uintptr_t lo = 0, hi = ~(uintptr_t)0;
      if (at_end(mine_row)) bounds(base[n], mine_row, lo, hi);
      const bool cut = lo > at || hi < at + row_bytes;  // some of the row is not in the copy
#pragma unroll
      for (int i = 0; i < c.NV; ++i) {
        v[i].clear();
        if (!c.any(i)) continue;
        if (c.whole(i) && !cut) {
          v[i].load(in + c.at(i));
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int col = c.at(i) + e;
            const uintptr_t mine = at + (long long)col * sizeof(T);
            if (c.has(i, e)) v[i].put_element(e, mine >= lo && mine < hi ? in[col] : src[col]);
          }
        }
      }
    }
  }
};

template <typename T, int VEC, int E, int OWN, bool EVEN>
__device__ __forceinline__ void write(T* out, const Raw<T, VEC>& v, int i, const Cols<VEC, E, OWN, EVEN>& c) {
  if (c.whole(i)) {
    if (c.any(i)) v.store(out + c.at(i));
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (c.has(i, e)) out[c.at(i) + e] = v.element(e);
    }
  }
}

// A vector of D weights as the threads' vectors read it: staged in shared
// memory with the block's shift (zero around the row), or in place.  Null: f.
template <typename WT, int VEC, int E, int OWN, bool EVEN>
struct Weights {
  using C = Cols<VEC, E, OWN, EVEN>;
  const WT* p;  // column 0
  static __host__ __device__ int bytes(int D) { return (D + 2 * 8) * (int)sizeof(WT) / 16 * 16 + 16; }
  __device__ __forceinline__ Weights(const WT* src, char*& dyn, const C& c) {
    p = src;
    if (!src || !kStaged<VEC, EVEN>) return;
    WT* q = reinterpret_cast<WT*>(dyn);
    dyn += bytes(c.D);
    const int span = (c.D + c.shift + VEC - 1) / VEC * VEC;
    for (int i0 = threadIdx.x; i0 < span; i0 += 8 * blockDim.x) {
      WT v[8];  // loads first: their latency would be paid one by one
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int col = i0 + u * (int)blockDim.x - c.shift;
        v[u] = (WT)0.f;
        if (col >= 0 && col < c.D) v[u] = src[col];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * (int)blockDim.x;
        if (i < span) q[i] = v[u];
      }
    }
    p = q + c.shift;
  }
  __device__ __forceinline__ void load(int i, Unit<VEC> (&u)[kUnits<VEC>], float f, const C& c) const {
    if (p) {
      Raw<WT, VEC> q;
      q.load(p + c.at(i));
#pragma unroll
      for (int j = 0; j < kUnits<VEC>; ++j) u[j] = q.unit(j);
    } else {
#pragma unroll
      for (int j = 0; j < kUnits<VEC>; ++j) u[j] = all<VEC>(f);
    }
  }
};

// Sums of K values over the threads of a row; every thread gets them.  The
// first exchanges halve the number of values a lane carries (lane groups end
// up with one value each), the rest add it up, and a last round hands them out:
// about 2 K shuffles instead of 5 K.  Blocks alternate between two buffers
// (flip), so one barrier per sum suffices: it also stands between a buffer's
// readers and its next writers.
template <int K, int OWN>
__device__ __forceinline__ void row_sum(float (&v)[K], int& flip) {
  constexpr int P = K <= 1 ? 1 : K <= 2 ? 2 : K <= 4 ? 4 : K <= 8 ? 8 : K <= 16 ? 16 : 32;
  constexpr int G = 32 / P;  // lanes per value
  const int lane = threadIdx.x & 31;
  float t[P];
#pragma unroll
  for (int k = 0; k < P; ++k) t[k] = k < K ? v[k < K ? k : 0] : 0.f;
#pragma unroll
  for (int half = P / 2, mask = 16; half > 0; half /= 2, mask /= 2) {
    const bool up = lane & mask;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float send = up ? t[k] : t[k + half], keep = up ? t[k + half] : t[k];
      t[k] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
    }
  }
  float mine = t[0];  // the value with index lane / G
#pragma unroll
  for (int o = G / 2; o > 0; o /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if constexpr (OWN != kWarp) {
    __shared__ float part[2][16][P];
    const int w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    flip ^= 1;
    if (lane % G == 0) part[flip][w][lane / G] = mine;
    __syncthreads();
    mine = 0.f;
    for (int i = lane % G; i < nw; i += G) mine += part[flip][i][lane / G];
#pragma unroll
    for (int o = G / 2; o > 0; o /= 2) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = P == 1 ? mine : __shfl_sync(0xffffffffu, mine, k * G);
}

// Each block adds up its rows' contributions to N column sums in registers
// (acc); this writes the block's own totals to out[n][D] (null: not wanted),
// summed over its warps in a fixed order.  sh: N x kWarps x D floats (unused when
// a block owns a row).
template <int N, int VEC, int E, int OWN, bool EVEN>
__device__ __forceinline__ void write_column_sums(const Unit<VEC> (&acc)[N][E / VEC][kUnits<VEC>],
                                                  float* const (&out)[N], float* sh,
                                                  const Cols<VEC, E, OWN, EVEN>& c) {
  if (OWN == kWarp) __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!out[n]) continue;
    float* to = OWN != kWarp ? out[n] : sh + (n * kWarps + (threadIdx.x >> 5)) * c.D;
#pragma unroll
    for (int i = 0; i < c.NV; ++i) {
#pragma unroll
      for (int j = 0; j < kUnits<VEC>; ++j) {
        if constexpr (VEC == 1) {
          if (c.any(i)) to[c.at(i)] = acc[n][i][0];
        } else {
          const float2 f = row::parts(acc[n][i][j]);
          if constexpr (EVEN) {
            if (c.any(i)) *reinterpret_cast<float2*>(to + c.at(i) + 2 * j) = f;
          } else {
            if (c.has(i, 2 * j)) to[c.at(i) + 2 * j] = f.x;
            if (c.has(i, 2 * j + 1)) to[c.at(i) + 2 * j + 1] = f.y;
          }
        }
      }
    }
  }
  if constexpr (OWN == kWarp) {
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (!out[n]) continue;
      for (int col = threadIdx.x; col < c.D; col += blockDim.x) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += sh[(n * kWarps + w) * c.D + col];
        out[n][col] = t;
      }
    }
  }
}

// --- launches ---------------------------------------------------------------------------------------

// How a launch reads its rows: whole vectors (vec), of rows that repeat their
// place against 16-byte bounds every `period` rows.
struct Layout {
  bool vec, even;
  int period, span;  // columns that a row's vectors cover
};
template <typename T>
inline Layout layout(int D, std::initializer_list<const void*> tensors, std::initializer_list<const void*> weights) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(*tensors.begin()) & 15;
  bool same = true;  // the optional ones may be null
  for (const void* p : tensors) same = same && (!p || (reinterpret_cast<uintptr_t>(p) & 15) == at);
  const int bytes = D * (int)sizeof(T);
  // even rows read the weights in whole vectors from where they lie
  bool even = at == 0 && bytes % 16 == 0;
  for (const void* p : weights) even = even && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
  if (!same || (!even && D + row::kFull<T> > 4096)) return Layout{false, false, 1, D};
  int period = 1;
  while (period * bytes % 16 != 0) period *= 2;
  return Layout{true, even, period, even ? D : D + row::kFull<T> - 1};
}

// Elements per thread of rows that span `cols` columns.
inline int elements(int cols) {
  if (cols <= kWarpCols) return (cols + 255) / 256 * 8;
  return cols <= 8192 ? 16 : 32;
}

// `rows` rows, at most max_blocks blocks of 256 threads (or more, smaller ones)
// that walk over them.
struct Shape {
  int threads, blocks;
};
inline Shape shape(long long rows, const Layout& l, int max_blocks) {
  Shape s;
  const int e = elements(l.span);
  const bool block = l.span > kWarpCols;
  s.threads = block ? ((l.span + e - 1) / e + 31) / 32 * 32 : kWarps * 32;
  long long want = block ? rows : (rows + kWarps - 1) / kWarps;
  max_blocks *= blocks_per_max(s.threads);
  want = want < max_blocks ? want : max_blocks;
  s.blocks = (int)((want + l.period - 1) / l.period * l.period);
  return s;
}

// Calls f with the compile-time (VEC, E, OWN, EVEN) of a launch.
template <typename T, typename F>
inline void dispatch(const Layout& l, F&& f) {
  constexpr int V = row::kFull<T>;
  auto with = [&](auto e, auto own) {
    if (l.even) f(std::integral_constant<int, V>{}, e, own, std::true_type{});
    // tensors that are shifted differently: the widest kernel of a warp serves all its rows
    else if (!l.vec) f(std::integral_constant<int, 1>{}, std::integral_constant<int, own() == kWarp ? 32 : e()>{}, own,
                       std::false_type{});
    // rows off the bounds with more than 4096 columns never come as vectors
    else if constexpr (own() != kBlock512) f(std::integral_constant<int, V>{}, e, own, std::false_type{});
  };
  std::integral_constant<int, kWarp> warp;
  if (l.span > 8192) with(std::integral_constant<int, 32>{}, std::integral_constant<int, kBlock512>{});
  else if (l.span > 4096) with(std::integral_constant<int, 16>{}, std::integral_constant<int, kBlock512>{});
  else if (l.span > kWarpCols) with(std::integral_constant<int, 16>{}, std::integral_constant<int, kBlock256>{});
  else if (l.span > 768) with(std::integral_constant<int, 32>{}, warp);
  else if (l.span > 512) with(std::integral_constant<int, 24>{}, warp);
  else if (l.span > 256) with(std::integral_constant<int, 16>{}, warp);
  else with(std::integral_constant<int, 8>{}, warp);
}

// Ring depth of a launch, and its dynamic shared memory: the staged weights
// (nw vectors), then the ring or, after it, the warps' column sums.
template <typename T, typename WT, int N, int VEC, int E, int OWN, bool EVEN>
inline int ring_stages(int D, long long rows, const Layout& l, const Shape& sh, int nw, int sums, int* smem) {
  constexpr int R = kRows<T, E, N>;
  using G = Ring<T, N, R, VEC, OWN, EVEN>;
  const int fixed = kStaged<VEC, EVEN> ? nw * Weights<WT, VEC, E, OWN, EVEN>::bytes(D) : 0;
  const int per = G::kOwners * N * R * G::slot_bytes(D);
  int s = (kRingMemory / (kResident<T, E, OWN> * blocks_per_max(sh.threads)) - fixed) / per;
  if (s > kMaxStages) s = kMaxStages;
  const long long owners = (long long)sh.blocks * G::kOwners * R;
  const long long each = (rows + owners - 1) / owners;
  if (s > each) s = (int)each;
  if (s < 1) s = 1;
  const int need = OWN == kWarp ? sums * kWarps * D * (int)sizeof(float) : 0;
  *smem = fixed + (s * per > need ? s * per : need);
  return s;
}

// Launches one of the kernels with `smem` bytes of dynamic shared memory.
template <typename... P, typename... A>
inline cudaError_t launch_rows(void (*kernel)(P...), const Shape& sh, int smem, cudaStream_t s, A... args) {
  if (smem > kDynamicMemory) return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamicMemory);
  return e != cudaSuccess ? e : chained(kernel, dim3(sh.blocks), dim3(sh.threads), smem, 1, s, args...);
}

// Blocks of 256 threads of the kernels that reduce over rows (one partial sum
// row each): two per multiprocessor of a GB300, in whole periods.  A constant,
// so that the workspace depends on the sizes alone.
constexpr int kMaxParts = 304;

// Adds up `parts` partial rows in[k][parts][D] into out_k[D] (k < n).
cudaError_t reduce_parts(const float* in, int parts, int D, void* out0, void* out1, bool out_bf16, cudaStream_t s);

}  // namespace ln
}  // namespace fbob
