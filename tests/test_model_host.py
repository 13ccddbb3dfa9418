"""Host-side refusals of the operators around the attention (no GPU: every
check precedes the first CUDA call)."""

import ctypes

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from exact_second_order_attn_gb300 import _lib
from exact_second_order_attn_gb300.build import build

INVALID, UNSUPPORTED, WORKSPACE = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def rotary_call(lib, r, B=1, N=4, d=8, dtype=0, H=2, count=1, x=0x1000, y=0x2000, xs=None, ys=None, positions=None,
                size=8, step=0):
    t = (_lib.RotaryHeads * 2)()
    for e in t:
        e.x, e.y, e.H = x, y, H
        e.x_stride[:] = xs or (H * N * d, N * d, d)
        e.y_stride[:] = ys or (H * N * d, N * d, d)
    return lib.fbob_rotary_apply(ctypes.byref(r) if r else None, B, N, d, dtype, t if count else None, count, positions,
                                 size, step, 0, 0, None)


@pytest.mark.parametrize("field,value,status", [
    ("rot", 0, INVALID), ("rot", -2, INVALID), ("rot", 7, INVALID), ("rot", 258, UNSUPPORTED), ("rot", 10, INVALID),
    ("base", 1.0, INVALID), ("base", float("nan"), INVALID), ("base", float("inf"), INVALID),
    ("magnitude", 0.0, INVALID), ("magnitude", float("inf"), INVALID), ("scaling", 4, INVALID), ("scaling", -1, INVALID),
])
def test_rotary_description_refusals(lib, field, value, status):
    r = fb.Rotary(8)
    setattr(r, field, value)
    assert rotary_call(lib, r) == status


@pytest.mark.parametrize("kw,status", [
    (dict(scaling="linear", factor=0.5), INVALID), (dict(scaling="linear", factor=float("nan")), INVALID),
    (dict(scaling="parts", factor=2.0), INVALID), (dict(scaling="parts", factor=2.0, original=-1.0), INVALID),
    (dict(scaling="parts", factor=2.0, original=9.0, slow=4.0, fast=4.0), INVALID),
    (dict(scaling="parts", factor=2.0, original=9.0, slow=-1.0), INVALID),
])
def test_rotary_scaling_refusals(lib, kw, status):
    assert rotary_call(lib, fb.Rotary(8, **kw)) == status
    assert rotary_call(lib, fb.Rotary(2, scaling="base", factor=2.0)) == INVALID
    with pytest.raises(ValueError):
        fb.Rotary(8, scaling="other")


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(d=0), INVALID), (dict(d=257), UNSUPPORTED), (dict(d=6), INVALID),
    (dict(dtype=9), INVALID), (dict(count=0), INVALID), (dict(count=3), INVALID), (dict(H=-1), INVALID),
    (dict(H=70000), UNSUPPORTED), (dict(B=70000, N=70000), UNSUPPORTED), (dict(x=0), INVALID), (dict(y=0), INVALID),
    (dict(x=0x1001), INVALID), (dict(y=0x2002, dtype=1), INVALID), (dict(xs=(-8, 8, 8)), INVALID),
    (dict(ys=(64, 32, -8)), INVALID), (dict(ys=(64, 32, 0)), INVALID), (dict(ys=(64, 32, 7)), INVALID),
    (dict(ys=(64, 0, 8)), INVALID), (dict(ys=(0, 32, 8), B=2), INVALID), (dict(ys=(56, 32, 8), B=2), INVALID),
    (dict(positions=0x3001), INVALID), (dict(positions=0x3000, size=2), INVALID),
    (dict(positions=0x3000, step=-1), INVALID),
])
def test_rotary_call_refusals(lib, kw, status):
    assert rotary_call(lib, fb.Rotary(8), **kw) == status


def test_rotary_empty_problems_and_null(lib):
    for kw in (dict(B=0), dict(N=0), dict(H=0)):
        assert rotary_call(lib, fb.Rotary(8), **kw) == _lib.OK
    assert rotary_call(lib, None) == INVALID
    assert lib.fbob_rotary_frequencies(ctypes.byref(fb.Rotary(8)), None) == INVALID


def norm_calls(lib, p, ptr=0x1000, ws=0x9000, ws_bytes=None, drop=None):
    ref = ctypes.byref(p) if p else None
    if ws_bytes is None:
        ws_bytes = lib.fbob_layer_norm_workspace_bytes(ref) if p else 0
    def ptrs(n):
        return [None if i == drop else ptr for i in range(n)]
    return (lib.fbob_layer_norm_fwd(ref, *ptrs(6), None), lib.fbob_layer_norm_bwd(ref, *ptrs(8), ws, ws_bytes, None),
            lib.fbob_layer_norm_bob(ref, *ptrs(11), ws, ws_bytes, None))


def norm(rows=4, D=64, dtype=_lib.BF16, wtype=_lib.FP32, eps=1e-5):
    return _lib.Norm(rows, D, dtype, wtype, eps)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(D=-3), INVALID), (dict(D=16385), UNSUPPORTED),
    (dict(rows=2 ** 40), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(wtype=5), INVALID),
    (dict(dtype=_lib.FP32, wtype=_lib.BF16), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
])
def test_norm_descriptor_refusals(lib, kw, status):
    assert norm_calls(lib, norm(**kw)) == (status,) * 3


def test_norm_pointer_and_workspace_refusals(lib):
    assert norm_calls(lib, None) == (INVALID,) * 3
    assert norm_calls(lib, norm(), ptr=0x1001) == (INVALID,) * 3
    assert norm_calls(lib, norm(), drop=0) == (INVALID,) * 3
    assert norm_calls(lib, norm(), ws=0)[1:] == (WORKSPACE,) * 2
    assert norm_calls(lib, norm(), ws=0x9004)[1:] == (WORKSPACE,) * 2
    p = norm()
    need = lib.fbob_layer_norm_workspace_bytes(ctypes.byref(p))
    assert norm_calls(lib, p, ws_bytes=need - 1)[1] == WORKSPACE
    assert norm_calls(lib, p, ws_bytes=need // 2 - 1)[1:] == (WORKSPACE,) * 2
    assert lib.fbob_layer_norm_workspace_bytes(None) == 0
    # nothing asked for, nothing launched
    x = ctypes.c_void_p(0x1000)
    assert lib.fbob_layer_norm_bwd(ctypes.byref(p), x, x, x, x, x, None, None, None, None, 0, None) == _lib.OK
    assert lib.fbob_layer_norm_bob(ctypes.byref(p), x, x, x, x, x, x, x, x, None, None, None, None, 0, None) == _lib.OK


def test_binding_refuses_host_tensors_types_and_shapes():
    x = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError):
        fb.fbob_rotary_apply(fb.Rotary(8), x)
    with pytest.raises(ValueError):
        fb.fbob_rotary_apply(fb.Rotary(8), x[0])
    with pytest.raises(ValueError):
        fb.fbob_layer_norm_fwd(x)
    with pytest.raises(TypeError):
        fb.fbob_layer_norm_fwd(x.half())
    with pytest.raises(ValueError):
        fb.layer_norm(x.transpose(0, 1))


def ce(T=4, D=64, V=50, dtype=_lib.BF16, ignore=-100, piece=0):
    return _lib.LinearCe(T, D, V, dtype, ignore, piece)


def ce_calls(lib, p, ptr=0x1000, drop=None, ws=0x100000, short=0):
    ref = ctypes.byref(p) if p else None
    def ptrs(n):
        return [None if i == drop else ptr for i in range(n)]
    def size(which):
        return max(0, lib.fbob_linear_ce_workspace_bytes(ref, which) - short) if p else 0
    return (lib.fbob_linear_ce_fwd(ref, *ptrs(5), ws, size(0), None),
            lib.fbob_linear_ce_bwd(ref, *ptrs(7), ws, size(1), None),
            lib.fbob_linear_ce_bob(ref, *ptrs(10), ws, size(2), None))


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(V=0), INVALID), (dict(V=-5), INVALID), (dict(piece=-1), INVALID),
    (dict(dtype=3), INVALID), (dict(T=2 ** 24 + 1), UNSUPPORTED), (dict(V=2 ** 24 + 1), UNSUPPORTED),
    (dict(D=2 ** 15 + 1), UNSUPPORTED),
    (dict(T=2 ** 23, V=2 ** 23, D=8), UNSUPPORTED),
])
def test_linear_ce_descriptor_refusals(lib, kw, status):
    assert ce_calls(lib, ce(**kw)) == (status,) * 3
    assert lib.fbob_linear_ce_workspace_bytes(ctypes.byref(ce(**kw)), 1) == 0


def test_linear_ce_pointer_and_workspace_refusals(lib):
    assert ce_calls(lib, None) == (INVALID,) * 3
    assert ce_calls(lib, ce(), ptr=0x1001) == (INVALID,) * 3
    assert ce_calls(lib, ce(), ptr=0x1004) == (INVALID,) * 3   # W off 16 bytes, targets off 8
    for drop in range(5):
        assert ce_calls(lib, ce(), drop=drop) == (INVALID,) * 3
    assert ce_calls(lib, ce(), ws=0) == (WORKSPACE,) * 3
    assert ce_calls(lib, ce(), ws=0x100008) == (WORKSPACE,) * 3
    assert ce_calls(lib, ce(), short=1) == (WORKSPACE,) * 3
    assert lib.fbob_linear_ce_workspace_bytes(None, 0) == 0
    assert lib.fbob_linear_ce_workspace_bytes(ctypes.byref(ce()), 3) == 0
    # nothing asked for, nothing launched
    x, ref = ctypes.c_void_p(0x1000), ctypes.byref(ce())
    assert lib.fbob_linear_ce_bwd(ref, x, x, x, x, x, None, None, None, 0, None) == _lib.OK
    assert lib.fbob_linear_ce_bob(ref, x, x, x, x, x, x, x, None, None, None, None, 0, None) == _lib.OK
    assert lib.fbob_linear_ce_bob(ref, x, x, x, x, x, None, None, x, x, x, x, 0, None) == INVALID


def test_linear_ce_workspace_is_bounded_by_the_piece(lib):
    """The workspace holds a piece of the classes, not all of them."""
    def need(**kw):
        return lib.fbob_linear_ce_workspace_bytes(ctypes.byref(ce(**kw)), 1)
    big = dict(T=65536, D=64, V=200000)
    assert need(**big) < 65536 * 200000 * 2 / 20
    assert need(piece=256, **big) < need(piece=2048, **big) < need(**big)


def test_linear_ce_binding_refuses_shapes_and_types():
    H, W, y = torch.zeros(3, 8), torch.zeros(5, 8), torch.zeros(3, dtype=torch.int64)
    for h, w in ((H[0], W), (H, W[:, :4]), (H, W[0])):
        with pytest.raises(ValueError):
            fb.fbob_linear_ce_fwd(h, w, y)
    with pytest.raises(ValueError):
        fb.fbob_linear_ce_fwd(H, W, y)   # host tensors
    with pytest.raises(TypeError):
        fb.fbob_linear_ce_fwd(H.half(), W, y)
    with pytest.raises(ValueError):
        fb.linear_cross_entropy(H.t().contiguous().t(), W, y)
