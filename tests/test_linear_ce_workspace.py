"""Where the linear head's passes place their parts in a workspace: callers
may start it on any 16-byte bound, the kernels access it 32 bytes at a time."""

import ctypes

import pytest

from exact_second_order_attn_gb300 import _lib
from exact_second_order_attn_gb300.build import build
from native_helpers import compiled


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = compiled(str(tmp_path_factory.mktemp("ws")), """
        #include "ce.h"
        extern "C" unsigned long long base(unsigned long long ws) {
          return reinterpret_cast<uintptr_t>(fbob::ce::workspace_base(reinterpret_cast<void*>(ws)));
        }
        extern "C" unsigned long long slack() { return fbob::ce::kWorkspaceSlack; }
    """)
    for f in (lib.base, lib.slack):
        f.restype = ctypes.c_ulonglong
    lib.base.argtypes = [ctypes.c_ulonglong]
    return lib


def test_base_is_aligned_and_within_the_slack(host):
    for ws in range(1 << 20, (1 << 20) + 512, 16):
        base = host.base(ws)
        assert base % 256 == 0 and 0 <= base - ws <= host.slack()


@pytest.mark.parametrize("shape", [(1, 8, 1), (37, 65, 301), (24, 768, 5003), (8192, 768, 50257)])
@pytest.mark.parametrize("dtype", [_lib.BF16, _lib.FP32])
@pytest.mark.parametrize("which", [0, 1, 2])
def test_the_size_that_callers_are_told_holds_the_slack(host, shape, dtype, which):
    """The parts are whole multiples of 256 bytes; the slack comes on top."""
    build()
    need = _lib.load().fbob_linear_ce_workspace_bytes(ctypes.byref(_lib.LinearCe(*shape, dtype, -100, 0)), which)
    assert need % 256 == host.slack() and need > host.slack()


@pytest.mark.parametrize("T", [60000, 131072, 262144, 1 << 20])
@pytest.mark.parametrize("dtype", [_lib.BF16, _lib.FP32])
@pytest.mark.parametrize("which", [1, 2])
def test_the_classes_that_are_held_by_default(T, dtype, which):
    """As many as 512 MiB hold, but at least 2048, in equal pieces.  (One slab of
    dH's sums at this width, so that the piece alone changes the size.)"""
    build()

    def need(piece):
        return _lib.load().fbob_linear_ce_workspace_bytes(
            ctypes.byref(_lib.LinearCe(T, 2048, 128256, dtype, -100, piece)), which)

    terms = 3 if dtype == _lib.FP32 else 1
    room = (need(512) - need(256)) // 256  # bytes of a class
    assert T * 2 * terms * which <= room <= T * 2 * terms * which + 256
    cols = max(2048, (512 << 20) // room)
    cols = -(-128256 // -(-128256 // (-(-cols // 256) * 256)))
    cols = -(-cols // 256) * 256
    assert need(0) == need(256) + (cols - 256) * room
    assert cols * room <= max(512 << 20, 2048 * room) + 256 * room


@pytest.mark.parametrize("T,V,which", [(8192, 32768, 1), (4096, 32768, 2), (65536, 4096, 1), (131072, 2048, 1)])
def test_classes_that_just_fit_are_one_piece(T, V, which):
    """T x V x 2 bytes of 512 MiB: the second terms' rows of a few tokens do not
    make two pieces of them."""
    build()
    a, b = (_lib.load().fbob_linear_ce_workspace_bytes(ctypes.byref(_lib.LinearCe(T, 2048, V, _lib.BF16, -100, piece)),
                                                       which) for piece in (0, V))
    assert a == b
