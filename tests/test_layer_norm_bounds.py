"""The bounds of layer norm's bulk copies, restated: every copy is 16-byte
aligned, stays inside its tensor and its slot, and with the elements read
directly it covers the row."""

import pytest


def bounds(start, rows, row_bytes, r):
    at, end = start + r * row_bytes, start + rows * row_bytes
    lo = max(at & ~15, (start + 15) & ~15)
    hi = min((at + row_bytes + 15) & ~15, end & ~15)
    return at, lo, max(lo, hi)


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("D", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 769, 1537])
def test_copies_stay_inside_tensor_and_slot(size, D):
    slot = (D * size + 15) // 16 * 16 + 16
    for shift in range(0, 16, size):
        for rows in (1, 2, 3, 7, 20):
            start = 4096 + shift
            for r in range(rows):
                at, lo, hi = bounds(start, rows, D * size, r)
                assert lo % 16 == 0 and hi % 16 == 0 and lo <= hi
                if hi > lo:
                    assert start <= lo and hi <= start + rows * D * size
                    assert 0 <= lo - (at & ~15) and hi - (at & ~15) <= slot
                # an element inside the copy lies where the reader looks for it
                for j in (0, D // 2, D - 1):
                    mine = at + j * size
                    if lo <= mine < hi:
                        assert mine + size <= hi
                        assert (lo - (at & ~15)) + (mine - lo) == (at & 15) + j * size
