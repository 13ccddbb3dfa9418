// The dropout factor of an element from its place alone, so that no mask is
// stored: forward, gradients and the second order draw the same bits again.
//
// Philox4x32 in ten rounds (Salmon, Moraes, Dror, Shaw: Parallel Random Numbers:
// As Easy as 1, 2, 3, 2011): key = seed, counter = (column / 8, row, offset in 64
// bits).  Its four words serve eight neighbouring columns, sixteen bits each (low
// half first), since one word an element would double the generator's cost, which
// is issue: twenty wide products per call.  An element is dropped where its bits
// are below `dropped` of 65,536.
#pragma once

#include <stdint.h>

#include "internal.h"

namespace fbob {

struct Dropper {
  const uint32_t* keys;  // of the rounds, among the kernel's arguments: constants to the instructions
  uint32_t c2, c3;
  uint32_t last;  // 65536 dropped - 1: a half (in the upper bits) up to this is dropped
  float scale;
  bool on;

  // Reads the counter: after the kernel's dependencies.
  __device__ __forceinline__ explicit Dropper(const DropArgs& a) {
    on = a.dropped != 0;
    keys = a.keys;
    const unsigned long long at = a.offset + (on && a.counter ? (unsigned long long)*a.counter : 0ull);
    c2 = (uint32_t)at, c3 = (uint32_t)(at >> 32);
    last = (uint32_t)(a.dropped * 65536ull - 1ull);
    scale = a.scale;
  }

  __device__ __forceinline__ void words(uint32_t group, uint32_t row, uint32_t (&w)[4]) const {
    uint32_t a = group, b = row, c = c2, d = c3;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
      a = (uint32_t)(q >> 32) ^ b ^ keys[2 * i], b = (uint32_t)q;
      c = (uint32_t)(p >> 32) ^ d ^ keys[2 * i + 1], d = (uint32_t)p;
    }
    w[0] = a, w[1] = b, w[2] = c, w[3] = d;
  }

  // v[j] = m v[j] for columns 8 group + j of a row; what is dropped becomes 0
  // whatever it was.
  __device__ __forceinline__ void apply8(uint32_t group, uint32_t row, float* v) const {
    uint32_t w[4];
    words(group, row, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (j & 1 ? w[j / 2] : w[j / 2] << 16) > last ? v[j] * scale : 0.f;
  }
  // Bit j: column 8 group + j is kept.
  __device__ __forceinline__ uint32_t kept8(uint32_t group, uint32_t row) const {
    uint32_t w[4], k = 0;
    words(group, row, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) k |= (j & 1 ? w[j / 2] : w[j / 2] << 16) > last ? 1u << j : 0u;
    return k;
  }
  // The same as factors.
  __device__ __forceinline__ void factors8(uint32_t group, uint32_t row, float* m) const {
    uint32_t w[4];
    words(group, row, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = (j & 1 ? w[j / 2] : w[j / 2] << 16) > last ? scale : 0.f;
  }
};

}  // namespace fbob
