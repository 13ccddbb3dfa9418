// Rotary positions: y = m R(pos theta_i) x on pairs of the first `rot` columns
// of each head, the other columns copied; the transpose (the gradient's map)
// turns the other way.
//
// Angles.  The kernel holds each frequency as a 64-bit fixed-point fraction of
// a turn, F_i = theta_i / (2 pi) * 2^64, so pos * F_i mod 2^64 is the angle
// modulo a full turn with no range reduction.  What is left is theta_i's own
// rounding, below pos * 2^-52 radians (2e-10 at position 2^20, 5e-7 at 2^31, where
// it reaches an fp32 result's), and pos * 2^-64 turns from cutting F_i off.  The
// top 32 bits, read as a signed fraction x in [-1, 1) of half a turn, go to
// sincospif(x).
//
// Work split.  A thread owns one chunk of a token's head row (two vectors of
// VEC elements whose pairs it holds whole) and walks over a group of heads,
// so the sines are computed once for the group.  Bound by memory: every
// element is read once and written once.  2 x (16 + 16) heads of 16,384 x 128
// bf16, 537 MB: 85 us, 6.3 TB/s, 93 % of a measured copy.
#include <cuda_runtime.h>
#include <math.h>

#include "internal.h"
#include "prof.h"
#include "rowvec.cuh"

namespace fbob {
namespace {

using row::Raw;
constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads whose loads are issued together

template <typename T>
struct Side {
  const T* x;
  T* y;
  int H;
  long long xs[3], ys[3];
};

template <typename T>
struct Params {
  unsigned long long freq[kRotaryMaxPairs];
  Side<T> side[2];
  const void* positions;
  long long pos_stride, offset;
  int pos_bytes;  // 0: position = offset + n
  int N, d, rot;
  unsigned tokens, tokens_per_block;
  int chunks, rot_chunks, heads, group;
  float m, sign;
};

template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params<T> p) {
  const unsigned ti = threadIdx.x / (unsigned)p.chunks;
  const int chunk = (int)(threadIdx.x - ti * (unsigned)p.chunks);
  const unsigned long long token = (unsigned long long)blockIdx.x * p.tokens_per_block + ti;
  if (ti >= p.tokens_per_block || token >= p.tokens) return;
  const unsigned b = (unsigned)token / (unsigned)p.N;
  const int n = (int)((unsigned)token - b * (unsigned)p.N);

  const bool turn = chunk < p.rot_chunks;
  int o0, o1;
  if (turn) {
    o0 = IL ? chunk * 2 * VEC : chunk * VEC;
    o1 = IL ? o0 + VEC : o0 + (p.rot >> 1);
  } else {
    o0 = p.rot + (chunk - p.rot_chunks) * 2 * VEC;
    o1 = o0 + VEC;
  }
  const bool second = o1 < p.d;

  float c[VEC], s[VEC];
  if (turn) {
    long long pos = p.offset;
    const long long at = (long long)b * p.pos_stride + n;
    if (p.pos_bytes == 8) pos += reinterpret_cast<const long long*>(p.positions)[at];
    else if (p.pos_bytes == 4) pos += reinterpret_cast<const int*>(p.positions)[at];
    else pos += n;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const unsigned long long phase = (unsigned long long)pos * p.freq[chunk * VEC + j];
      sincospif((float)(int)(unsigned)(phase >> 32) * 0x1p-31f, &s[j], &c[j]);
      c[j] *= p.m;
      s[j] *= p.m * p.sign;
    }
  }

  const int h_end = min(((int)blockIdx.y + 1) * p.group, p.heads);
  for (int h0 = (int)blockIdx.y * p.group; h0 < h_end; h0 += kBatch) {
    Raw<T, VEC> a[kBatch], e[kBatch];
    T* out[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (h0 + k < h_end) {
        const int which = h0 + k >= p.side[0].H;
        const Side<T>& t = p.side[which];
        const int h = h0 + k - (which ? p.side[0].H : 0);
        const T* x = t.x + b * t.xs[0] + h * t.xs[1] + n * t.xs[2];
        out[k] = t.y + b * t.ys[0] + h * t.ys[1] + n * t.ys[2];
        a[k].load(x + o0);
        if (second) e[k].load(x + o1);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (h0 + k < h_end) {
        if (turn) {
          float u[2 * VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            // pair j of this chunk: the two halves' element j, or neighbours
            const float x0 = IL ? (2 * j < VEC ? a[k].get(2 * j) : e[k].get(2 * j - VEC)) : a[k].get(j);
            const float x1 = IL ? (2 * j + 1 < VEC ? a[k].get(2 * j + 1) : e[k].get(2 * j + 1 - VEC)) : e[k].get(j);
            u[IL ? 2 * j : j] = x0 * c[j] - x1 * s[j];
            u[IL ? 2 * j + 1 : VEC + j] = x0 * s[j] + x1 * c[j];
          }
          a[k].set(u);
          e[k].set(u + VEC);
        }
        a[k].store(out[k] + o0);
        if (second) e[k].store(out[k] + o1);
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RotaryArgs& a, cudaStream_t s) {
  constexpr int F = row::kFull<T>;
  Params<T> p;
  for (int i = 0; i < a.rot / 2; ++i) p.freq[i] = a.freq[i];
  // 16-byte vectors when every row of every tensor starts on 16 bytes and the
  // pairs and the unrotated rest divide into them; single elements otherwise.
  bool vec = a.rot % (2 * F) == 0 && a.d % F == 0;
  p.heads = 0;
  for (int k = 0; k < 2; ++k) {
    const RotarySide& t = a.side[k];
    p.side[k] = Side<T>{static_cast<const T*>(t.x), static_cast<T*>(t.y), t.H, {}, {}};
    for (int i = 0; i < 3; ++i) p.side[k].xs[i] = t.xs[i], p.side[k].ys[i] = t.ys[i];
    if (t.H == 0) continue;
    p.heads += t.H;
    vec = vec && ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y)) & 15u) == 0;
    for (int i = 0; i < 3; ++i) vec = vec && t.xs[i] % F == 0 && t.ys[i] % F == 0;
  }
  p.positions = a.positions;
  p.pos_stride = a.pos_stride;
  p.offset = a.offset;
  p.pos_bytes = a.positions ? a.pos_bytes : 0;
  p.N = a.N, p.d = a.d, p.rot = a.rot;
  p.tokens = (unsigned)a.B * (unsigned)a.N;
  const int v = vec ? F : 1;
  p.rot_chunks = a.rot / (2 * v);
  p.chunks = p.rot_chunks + (a.d - a.rot + 2 * v - 1) / (2 * v);
  p.tokens_per_block = kThreads / p.chunks;
  p.m = a.magnitude;
  p.sign = a.transpose ? -1.f : 1.f;
  const unsigned blocks = (p.tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  // Heads per thread: more share a thread's sines, fewer leave more blocks to
  // even out the last wave.  Eight at most (2 x 32 heads of 16,384 positions, half
  // of 128 columns rotated: 97 us with all 32, 87 with 8, 89 with 4), and as many
  // as leave the device four blocks per multiprocessor.
  p.group = p.heads < 8 ? p.heads : 8;
  while (p.group > 1 && (unsigned long long)blocks * ((p.heads + p.group - 1) / p.group) < 4ull * sm_count())
    p.group = (p.group + 1) / 2;
  const dim3 grid(blocks, (p.heads + p.group - 1) / p.group);
  prof_begin(s, "rotary");
  if (vec && a.interleaved) rotary_kernel<T, F, true><<<grid, kThreads, 0, s>>>(p);
  else if (vec) rotary_kernel<T, F, false><<<grid, kThreads, 0, s>>>(p);
  else if (a.interleaved) rotary_kernel<T, 1, true><<<grid, kThreads, 0, s>>>(p);
  else rotary_kernel<T, 1, false><<<grid, kThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t rotary(const RotaryArgs& a, cudaStream_t s) {
  return a.bf16 ? launch<row::bf16>(a, s) : launch<float>(a, s);
}

}  // namespace fbob
