"""The bounds of layer norm's bulk copies, by the kernels' own function on the
CPU: every copy is 16-byte aligned, stays inside its tensor and its slot, and
with the elements that are read directly it covers the row."""

import ctypes

import pytest

from native_helpers import compiled

SOURCE = """
#include "copy_bounds.h"
using namespace fbob::ln;
// 0, or the number of the first rule that a row of a tensor breaks.
extern "C" int check(unsigned long long start, long long rows, int row_bytes, int size, long long r) {
  const int edge = copy_edge(row_bytes), slot = (row_bytes + 15) / 16 * 16 + 16;
  const uintptr_t at = start + r * row_bytes, end = start + rows * row_bytes;
  uintptr_t lo, hi;
  copy_bounds(start, rows, row_bytes, edge, r, lo, hi);
  if (lo % 16 || hi % 16 || hi < lo) return 1;
  if (hi > lo && (lo < start || hi > end)) return 2;               // outside the tensor
  if (hi > lo && (lo < (at & ~(uintptr_t)15) || hi - (at & ~(uintptr_t)15) > (uintptr_t)slot)) return 3;  // the slot
  const bool cut = lo > at || hi < at + row_bytes;
  if (cut && !copy_at_end(r, rows, edge)) return 4;  // the reader would not look for missing elements
  for (int j = 0; j < row_bytes; j += size) {  // an element is in the copy whole or not at all
    const uintptr_t mine = at + j;
    if (mine >= lo && mine < hi && mine + size > hi) return 5;
    if (mine < lo && mine + size > lo && hi > lo) return 6;
  }
  // what is left out are the ends' 15 bytes at most
  if (hi > lo && (lo > at ? lo - at : 0) + (hi < at + row_bytes ? at + row_bytes - hi : 0) > 30) return 7;
  return 0;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = compiled(str(tmp_path_factory.mktemp("copies")), SOURCE)
    lib.check.argtypes = [ctypes.c_ulonglong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_longlong]
    return lib


@pytest.mark.parametrize("size", [2, 4])
def test_copies_stay_inside_tensor_and_slot(host, size):
    for D in [*range(1, 40), 769, 1537, 4095]:
        for shift in range(0, 16, size):
            for rows in (1, 2, 3, 7, 20, 40):
                for r in range(rows):
                    assert host.check(4096 + shift, rows, D * size, size, r) == 0, (D, shift, rows, r)


@pytest.mark.parametrize("D,size", [(1, 2), (3, 2), (769, 2), (1537, 4)])
def test_copies_of_rows_past_32_bits(host, D, size):
    rows = 2 ** 33 // D + 5
    for shift in range(0, 16, size):
        for r in (*range(20), rows // 2, *range(rows - 20, rows)):
            assert host.check((1 << 40) + shift, rows, D * size, size, r) == 0, (D, shift, r)
