// The bytes that layer norm's bulk copies bring for a row: 16-byte bounds around
// it, inside its tensor.  Host code too, so that it can be checked without a GPU.
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

namespace fbob {
namespace ln {

// Rows from a tensor's ends within which a row's bounds, moved outwards by up to
// 15 bytes, could pass them.
__host__ __device__ inline int copy_edge(int row_bytes) { return (15 + row_bytes) / row_bytes; }
__host__ __device__ inline bool copy_at_end(long long r, long long rows, int edge) {
  return r < edge || r >= rows - edge;
}

// Bounds of the copy for row r of the tensor of `rows` rows at `start`: the row's,
// moved outwards to 16 bytes, and inwards at the tensor's ends.  Empty if no whole
// 16 bytes are left.
__host__ __device__ inline void copy_bounds(uintptr_t start, long long rows, int row_bytes, int edge, long long r,
                                            uintptr_t& lo, uintptr_t& hi) {
  const uintptr_t at = start + r * row_bytes, mask = ~(uintptr_t)15;
  lo = at & mask;
  hi = (at + row_bytes + 15) & mask;
  if (copy_at_end(r, rows, edge)) {
    const uintptr_t first = (start + 15) & mask, last = (start + (uintptr_t)(rows * row_bytes)) & mask;
    lo = lo > first ? lo : first;
    hi = hi < last ? hi : last;
    if (hi < lo) hi = lo;
  }
}

}  // namespace ln
}  // namespace fbob
