"""The shared memory of layer norm's launches, by the library's own functions
on the CPU: every kernel has one allowance, and no launch asks for more."""

import ctypes

import pytest

from native_helpers import compiled

SOURCE = """
#include <initializer_list>
#include <type_traits>
#include "layer_norm.cuh"
using namespace fbob::ln;

// Bytes of a launch over N tensors at address x, weights at w.
template <typename T, typename WT, int N>
int bytes(int D, long long rows, unsigned long long x, unsigned long long w, int other, int nw, int sums) {
  const void *p = (const void*)x, *q = (const void*)(x + other * sizeof(T)), *v = (const void*)w;
  const Layout l = layout<T>(D, {p, q}, {v});
  const Shape sh = shape(rows, l, 304);
  int smem = -1;
  dispatch<T>(l, [&](auto vec, auto e, auto own, auto even) {
    ring_stages<T, WT, N, vec(), e(), own(), even()>(D, rows, l, sh, nw, sums, &smem);
  });
  return smem;
}
template <typename T, typename WT>
int pass(int which, int D, long long rows, unsigned long long x, unsigned long long w, int other) {
  if (which == 0) return bytes<T, WT, 1>(D, rows, x, w, other, 2, 0);
  if (which == 1) return bytes<T, WT, 2>(D, rows, x, w, other, 1, 2);
  return bytes<T, WT, 3>(D, rows, x, w, other, 3, 1);
}
extern "C" int allowance() { return kDynamicMemory; }
// Most bytes over all widths and a few row counts.
extern "C" int most(int type, int which, int shift, int other) {
  int top = -1;
  for (int D = 1; D <= 16384; ++D) {
    for (long long rows : {1ll, 40ll, 3000ll, 1000000ll}) {
      const unsigned long long x = 1 << 20, w = x + 4;
      for (unsigned long long at : {x, w}) {
        const int n = type == 0   ? pass<row::bf16, row::bf16>(which, D, rows, x + 2 * shift, at, other)
                      : type == 1 ? pass<row::bf16, float>(which, D, rows, x + 2 * shift, at, other)
                                  : pass<float, float>(which, D, rows, x + 4 * shift, at, other);
        if (n < 0) return 1 << 30;  // no kernel for this layout
        top = n > top ? n : top;
      }
    }
  }
  return top;
}
namespace fbob {
void prof_begin(cudaStream_t, const char*) {}
void prof_end(cudaStream_t) {}
int sm_count() { return 152; }
}  // namespace fbob
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("memory")), SOURCE.replace("row::bf16", "fbob::row::bf16"), nvcc=True)


@pytest.mark.parametrize("type_", [0, 1, 2])
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("shift,other", [(0, 0), (1, 0), (0, 1)])
def test_every_launch_is_within_the_allowance(host, type_, which, shift, other):
    # 227 KB a block, of which the kernels' static arrays take up to 4.2 KB
    assert 0 < host.most(type_, which, shift, other) <= host.allowance() <= 232448 - 4224
