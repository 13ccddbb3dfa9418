"""Host-side refusals of linear layers and dropout (no GPU: every check
precedes the first CUDA call)."""

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


def drop_call(lib, d, counter=None, rows=4, D=8, dtype=0, x=0x1000, r=None, y=0x2000):
    return lib.fbob_dropout_apply(ctypes.byref(d) if d else None, counter, rows, D, dtype, x, r, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(D=-8), INVALID), (dict(dtype=2), INVALID),
    (dict(rows=1 << 32), UNSUPPORTED), (dict(rows=1 << 30, D=1 << 11), UNSUPPORTED),
    (dict(D=(1 << 30) + 1), UNSUPPORTED), (dict(x=0), INVALID), (dict(y=0), INVALID), (dict(x=0x1001), INVALID),
    (dict(r=0x1001), INVALID), (dict(y=0x2002, dtype=1), INVALID), (dict(counter=0x1004), INVALID),
])
def test_dropout_refusals(lib, kw, status):
    assert drop_call(lib, fb.Dropout(0.5), **kw) == status


@pytest.mark.parametrize("p", [-0.1, 1.1, float("nan"), float("inf")])
def test_dropout_description_refusals(lib, p):
    assert drop_call(lib, fb.Dropout(p)) == INVALID
    assert drop_call(lib, None) == INVALID
    assert drop_call(lib, fb.Dropout(0.5), rows=0) == _lib.OK
    l = _lib.Linear(40, 8, 8, 0, 0)
    assert lib.fbob_linear_workspace_bytes(ctypes.byref(l), ctypes.byref(fb.Dropout(p)), 1) == 0


def linear_calls(lib, l, ptr=None, ws=0x9000, ws_bytes=None, drop=None, counter=None):
    """The statuses of the three calls; `ptr` replaces some addresses."""
    a = dict(x=0x1000, W=0x1000, b=0x1000, r=0x1000, y=0x2000, z=0x3000, dy=0x1000, ux=0x1000, uW=0x1000, ub=0x1000,
             dx=0x2000, dW=0x2000, db=0x2000, gx=0x2000, gW=0x2000, gb=0x2000, gdy=0x2000)
    a.update(ptr or {})
    p, d = ctypes.byref(l) if l else None, ctypes.byref(drop) if drop else None
    n = [lib.fbob_linear_workspace_bytes(p, d, i) if ws_bytes is None else ws_bytes for i in range(3)]
    names = (("x", "W", "b", "r", "y", "z"), ("x", "W", "z", "dy", "dx", "dW", "db"),
             ("x", "W", "z", "dy", "ux", "uW", "ub", "gx", "gW", "gb", "gdy"))
    calls = (lib.fbob_linear_fwd, lib.fbob_linear_bwd, lib.fbob_linear_bob)
    return [f(p, d, counter, *(a[k] for k in ks), ws, b, None) for f, ks, b in zip(calls, names, n)]


@pytest.mark.parametrize("field,value,status", [
    ("T", -1, INVALID), ("K", 0, INVALID), ("N", 0, INVALID), ("K", -8, INVALID), ("dtype", 7, INVALID),
    ("activation", 5, INVALID), ("activation", -1, INVALID), ("T", (1 << 24) + 1, UNSUPPORTED),
    ("K", (1 << 20) + 1, UNSUPPORTED), ("N", (1 << 20) + 1, UNSUPPORTED),
])
def test_linear_description_refusals(lib, field, value, status):
    l = _lib.Linear(40, 64, 64, 0, 2)
    setattr(l, field, value)
    assert linear_calls(lib, l) == [status] * 3
    assert lib.fbob_linear_workspace_bytes(ctypes.byref(l), None, 1) == 0


def test_linear_sizes_together(lib):
    assert linear_calls(lib, _lib.Linear(1 << 24, 1 << 17, 8, 0, 0)) == [UNSUPPORTED] * 3
    assert linear_calls(lib, _lib.Linear(1 << 24, 8, 1 << 17, 0, 0)) == [UNSUPPORTED] * 3
    assert linear_calls(lib, None) == [INVALID] * 3


@pytest.mark.parametrize("name,value,want", [
    ("x", 0, (1, 1, 1)), ("W", 0, (1, 1, 1)), ("y", 0, (1, 0, 0)), ("dy", 0, (0, 1, 1)), ("z", 0, (0, 1, 1)),
    ("x", 0x1008, (1, 1, 1)), ("W", 0x1002, (1, 1, 1)), ("dy", 0x1008, (0, 1, 1)), ("ux", 0x1008, (0, 0, 1)),
    ("uW", 0x1008, (0, 0, 1)), ("b", 0x1001, (1, 0, 0)), ("r", 0x1001, (1, 0, 0)), ("z", 0x3001, (1, 1, 1)),
    ("dx", 0x2001, (0, 1, 0)), ("gdy", 0x2001, (0, 0, 1)), ("ub", 0x2001, (0, 0, 1)),
])
def test_linear_pointer_refusals(lib, name, value, want):
    """With a workspace of no bytes the calls that accept the pointers fail there."""
    got = linear_calls(lib, _lib.Linear(40, 64, 63 if name in "y" else 64, 0, 2), {name: value}, ws_bytes=0)
    for st, w, i in zip(got, want, range(3)):
        if w:
            assert st == INVALID, i
        else:
            assert st != INVALID, i


def test_linear_workspace_and_absent_cotangents(lib):
    l = _lib.Linear(40, 64, 64, 1, 2)
    assert linear_calls(lib, l, ws=None) == [WORKSPACE] * 3
    assert linear_calls(lib, l, ws=0x9008) == [WORKSPACE] * 3
    need = [lib.fbob_linear_workspace_bytes(ctypes.byref(l), None, i) for i in range(3)]
    assert all(n > 0 for n in need)
    assert linear_calls(lib, l, ws_bytes=min(need) - 1)[0] == WORKSPACE
    assert linear_calls(lib, l, dict(ux=0, uW=0))[2] == INVALID
    assert linear_calls(lib, l, counter=0x1000) == [INVALID] * 3  # a counter without a dropout
    assert lib.fbob_linear_workspace_bytes(ctypes.byref(l), None, 3) == 0
    few = _lib.Linear(16, 64, 64, 1, 2)
    assert lib.fbob_linear_workspace_bytes(ctypes.byref(few), None, 0) == 0


def test_no_tokens_and_no_outputs(lib):
    none = {k: 0 for k in ("x", "W", "z", "dy", "dx", "dW", "db", "gx", "gW", "gb", "gdy", "y")}
    assert linear_calls(lib, _lib.Linear(0, 64, 64, 0, 2), none) == [_lib.OK] * 3
    quiet = {k: 0 for k in ("dx", "dW", "db", "gx", "gW", "gb", "gdy")}
    assert linear_calls(lib, _lib.Linear(40, 64, 64, 0, 2), quiet, ws_bytes=0)[1:] == [_lib.OK] * 2


@pytest.mark.parametrize("T,K,N", [(17, 8, 8), (40, 65, 301), (8192, 768, 2304), (1 << 24, 8, 16), (32, 1 << 20, 1 << 20)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspaces_hold_their_parts(lib, T, K, N, dtype):
    """Multiples of 256 bytes and the slack for the base; at least dz and q."""
    l = _lib.Linear(T, K, N, dtype, 2)
    for i in range(3):
        n = lib.fbob_linear_workspace_bytes(ctypes.byref(l), None, i)
        assert n % 256 in (0, 240)
        if i:
            assert n >= i * T * N * 2 * (3 if dtype else 1)


def test_binding_refusals(lib):
    fb._model._bind()
    x, W = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="CUDA"):
        fb.fbob_linear_fwd(x, W)
    with pytest.raises(ValueError, match="CUDA"):
        fb.fbob_dropout_apply(fb.Dropout(0.5), x)
    with pytest.raises(ValueError, match="activation"):
        fb.fbob_linear_fwd(x, W, activation="tanh")
    with pytest.raises(ValueError, match="needed"):
        fb.fbob_linear_fwd(x, W.T)
    with pytest.raises(TypeError):
        fb.fbob_linear_fwd(x.double(), W.double())
    with pytest.raises(TypeError):
        fb.fbob_dropout_apply(None, x)
    with pytest.raises(TypeError):
        fb.fbob_dropout_apply(fb.Rotary(8), x)
    with pytest.raises(ValueError, match="contiguous"):
        fb.linear(x.T, W)
    with pytest.raises(ValueError, match="contiguous"):
        fb.dropout(fb.Dropout(0.5), x.T)
    l = fb.linear_for(x, W, "gelu")
    assert (l.T, l.K, l.N, l.activation) == (4, 8, 6, 2)
    with pytest.raises(ValueError):
        fb.linear_for(x, W.T)


def test_a_stream_of_another_device_is_refused():
    import types
    s = types.SimpleNamespace(device=torch.device("cuda", 1))
    x, W = torch.zeros(4, 8), torch.zeros(6, 8)
    for call in (lambda: fb.fbob_linear_fwd(x, W, stream=s), lambda: fb.fbob_dropout_apply(fb.Dropout(0.5), x, stream=s),
                 lambda: fb.fbob_linear_bwd(x, W, None, x, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call()
