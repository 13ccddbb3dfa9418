"""ctypes binding of the operators around the attention: argument marshalling
only, like ``_lib`` (include/fbob.h has each call's contract).

The calls run on the device of their tensors, on ``stream`` or that device's
current stream; outputs and workspaces that are not given come from torch's
allocator on that stream.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from ._lib import LinearCe, Norm, Rotary, _check, load

DTYPES = {torch.bfloat16: _lib.BF16, torch.float32: _lib.FP32}


# The stream handle itself, without a Stream object around it (a call of the
# smallest sizes is bound by the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dtype(t):
    try:
        return DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _device(t, name):
    """The index of the CUDA device that the call runs on."""
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device")
    return index


def _tensor(t, name, index, dtype, shape=None):
    """Check one contiguous tensor argument (None passes)."""
    if t is None:
        return
    if t.get_device() != index:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _p(t):
    return None if t is None else t.data_ptr()


def _run(fn, index, stream, *args):
    """Call a launching entry point with device ``index`` current."""
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if status:
        _check(status)


def _new(like, shape, dtype, stream):
    """An uninitialised tensor of ``stream``'s pool (memory that other streams
    may still be using is not handed to it)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _out(given, name, like, index, shape, dtype, stream):
    """The given output, checked, or a new one."""
    if given is None:
        return _new(like, shape, dtype, stream)
    _tensor(given, name, index, dtype, shape)
    return given


# --- rotary positions -----------------------------------------------------------------------------

def fbob_rotary_frequencies(rotary: Rotary) -> list:
    """theta_i of the description, scaled (i < rot/2)."""
    out = (ctypes.c_double * max(1, rotary.rot // 2))()
    _check(load().fbob_rotary_frequencies(ctypes.byref(rotary), out))
    return list(out)


# fbob_rotary_heads as the library lays it out (the fields of RotaryHeads)
_HEADS = struct.Struct("@PPi6q")


def _heads(t, name, like, index):
    if t.get_device() != index:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device")
    if t.dtype != like.dtype:
        raise TypeError(f"{name}: expected {like.dtype}, got {t.dtype}")
    st = t.stride()
    if len(st) != 4:
        raise ValueError(f"{name} must be [B, H, N, d]")
    if st[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}: the columns of a head must be contiguous")
    return st


def _rotary_side(x, y, name, like, index, stream):
    """(description for the library, output) of one tensor."""
    xs, shape = _heads(x, name, like, index), x.shape
    if y is None:
        y = _new(like, shape, like.dtype, stream)
        ys = y.stride()
    else:
        ys = _heads(y, name + "o", like, index)
        if y.shape != shape:
            raise ValueError(f"{name}o: expected shape {tuple(shape)}, got {tuple(y.shape)}")
    return _HEADS.pack(x.data_ptr(), y.data_ptr(), shape[1], xs[0], xs[1], xs[2], ys[0], ys[1], ys[2]), y


def fbob_rotary_apply(rotary, Q, K=None, positions=None, offset=0, transpose=False, Qo=None, Ko=None, stream=None):
    """Rotary positions on Q [B, H, N, d] and K [B, Hk, N, d] (any strides over
    contiguous rows) in one launch: (Qo, Ko), or Qo alone without K; contiguous
    [B, H, N, d] if not given.  ``positions``: int32 or int64, [N] or [B, N],
    added to ``offset``; without them token n has position offset + n.
    ``transpose``: the map's transpose (gradients)."""
    if Q.dim() != 4:
        raise ValueError("Q must be [B, H, N, d]")
    dt, index = _dtype(Q), _device(Q, "Q")
    B, _, N, d = Q.shape
    side, Qo = _rotary_side(Q, Qo, "Q", Q, index, stream)
    if K is None:
        if Ko is not None:
            raise ValueError("Ko without K")
        sides, count = side, 1
    else:
        if K.dim() != 4 or K.shape[0] != B or K.shape[2] != N or K.shape[3] != d:
            raise ValueError(f"K: expected shape ({B}, Hk, {N}, {d}), got {tuple(K.shape)}")
        other, Ko = _rotary_side(K, Ko, "K", Q, index, stream)
        sides, count = side + other, 2
    at, size, step = None, 0, 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        if positions.get_device() != index:
            raise ValueError("positions: all tensors must be on the same CUDA device")
        if positions.shape != (N,) and positions.shape != (B, N):
            raise ValueError(f"positions: expected shape ({N},) or ({B}, {N}), got {tuple(positions.shape)}")
        st = positions.stride()
        if st[-1] != 1 and N > 1:
            raise ValueError("positions must be contiguous")
        at, size = positions.data_ptr(), positions.element_size()
        step = st[0] if len(st) == 2 and B > 1 else 0
    _run(load().fbob_rotary_apply, index, stream, rotary, B, N, d, dt, sides, count, at, size, step, int(offset),
         int(bool(transpose)))
    return Qo if K is None else (Qo, Ko)


# --- layer norm -----------------------------------------------------------------------------------

def norm_for(x: torch.Tensor, weight_dtype: torch.dtype, eps: float = 0.0) -> Norm:
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    if weight_dtype not in DTYPES:
        raise TypeError(f"unsupported dtype {weight_dtype}")
    D = x.shape[-1]
    return Norm(x.numel() // D if D else 0, D, _dtype(x), DTYPES[weight_dtype], float(eps))


def fbob_layer_norm_workspace_bytes(p: Norm) -> int:
    return int(load().fbob_layer_norm_workspace_bytes(ctypes.byref(p)))


def _weight_dtype(x, *ws):
    for w in ws:
        if w is not None:
            return w.dtype
    return x.dtype


def _floats(workspace, need, x, index, stream):
    """(pointer, bytes) of the given fp32 workspace or of a new one."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _new(x, ((need + 3) // 4,), torch.float32, stream)
    else:
        _tensor(workspace, "workspace", index, torch.float32)
    return workspace.data_ptr(), workspace.numel() * 4, workspace


def fbob_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """(y, mean, rstd) = layer norm over the last dimension of x (contiguous,
    any leading shape); mean and rstd are fp32 of the leading shape."""
    wt = _weight_dtype(x, weight, bias)
    p, index = norm_for(x, wt, eps), _device(x, "x")
    shape = x.shape
    rows, cols = shape[:-1], shape[-1:]
    _tensor(x, "x", index, x.dtype)
    _tensor(weight, "weight", index, wt, cols)
    _tensor(bias, "bias", index, wt, cols)
    y = _out(y, "y", x, index, shape, x.dtype, stream)
    mean = _out(mean, "mean", x, index, rows, torch.float32, stream)
    rstd = _out(rstd, "rstd", x, index, rows, torch.float32, stream)
    _run(load().fbob_layer_norm_fwd, index, stream, p, x.data_ptr(), _p(weight), _p(bias), y.data_ptr(),
         mean.data_ptr(), rstd.data_ptr())
    return y, mean, rstd


def _norm_common(x, weight, mean, rstd, dy, index):
    shape = x.shape
    _tensor(x, "x", index, x.dtype)
    _tensor(mean, "mean", index, torch.float32, shape[:-1])
    _tensor(rstd, "rstd", index, torch.float32, shape[:-1])
    _tensor(dy, "dy", index, x.dtype, shape)
    if weight is not None:
        _tensor(weight, "weight", index, weight.dtype, shape[-1:])
    return shape, shape[-1:]


def fbob_layer_norm_bwd(x, weight, mean, rstd, dy, dx=None, dw=None, db=None, want=(True, True, True),
                        bias_dtype=None, workspace=None, stream=None):
    """(dx, dw, db) = layer norm's backward; ``want`` says which to compute
    (the others are None).  dw needs ``weight``; without one db has
    ``bias_dtype`` (default: x's)."""
    wt = weight.dtype if weight is not None else bias_dtype or x.dtype
    p, index = norm_for(x, wt), _device(x, "x")
    shape, cols = _norm_common(x, weight, mean, rstd, dy, index)
    want = (want[0], want[1] and weight is not None, want[2])
    dx = _out(dx, "dx", x, index, shape, x.dtype, stream) if want[0] else None
    dw = _out(dw, "dw", x, index, cols, wt, stream) if want[1] else None
    db = _out(db, "db", x, index, cols, wt, stream) if want[2] else None
    lib, need = load(), 0
    if want[1] or want[2]:
        need = lib.fbob_layer_norm_workspace_bytes(p) // (1 if want[1] and want[2] else 2)
    at, size, workspace = _floats(workspace, need, x, index, stream)
    _run(lib.fbob_layer_norm_bwd, index, stream, p, x.data_ptr(), _p(weight), mean.data_ptr(), rstd.data_ptr(),
         dy.data_ptr(), _p(dx), _p(dw), _p(db), at, size)
    return dx, dw, db


def fbob_layer_norm_bob(x, weight, mean, rstd, dy, ux, uw=None, ub=None, gx=None, gw=None, gdy=None,
                        want=(True, True, True), workspace=None, stream=None):
    """(gx, gw, gdy) = the vector-Jacobian product of layer norm's backward
    along (ux, uw, ub); ``want`` says which to compute.  gw needs ``weight``."""
    wt = _weight_dtype(x, weight, uw, ub)
    p, index = norm_for(x, wt), _device(x, "x")
    shape, cols = _norm_common(x, weight, mean, rstd, dy, index)
    _tensor(ux, "ux", index, x.dtype, shape)
    _tensor(uw, "uw", index, wt, cols)
    _tensor(ub, "ub", index, wt, cols)
    want = (want[0], want[1] and weight is not None, want[2])
    gx = _out(gx, "gx", x, index, shape, x.dtype, stream) if want[0] else None
    gw = _out(gw, "gw", x, index, cols, wt, stream) if want[1] else None
    gdy = _out(gdy, "gdy", x, index, shape, x.dtype, stream) if want[2] else None
    lib = load()
    need = lib.fbob_layer_norm_workspace_bytes(p) // 2 if want[1] else 0
    at, size, workspace = _floats(workspace, need, x, index, stream)
    _run(lib.fbob_layer_norm_bob, index, stream, p, x.data_ptr(), _p(weight), mean.data_ptr(), rstd.data_ptr(),
         dy.data_ptr(), ux.data_ptr(), _p(uw), _p(ub), _p(gx), _p(gw), _p(gdy), at, size)
    return gx, gw, gdy


# --- cross entropy of a linear head -----------------------------------------------------------------

def linear_ce_for(H: torch.Tensor, W: torch.Tensor, ignore_index: int = -100, piece: int = 0) -> LinearCe:
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError(f"H [T, D] and W [V, D] are needed, got {tuple(H.shape)} and {tuple(W.shape)}")
    (T, D), V = H.shape, W.shape[0]
    if max(T, D, V) > 2 ** 31 - 1:
        raise ValueError("sizes must fit 32 bits")
    return LinearCe(T, D, V, _dtype(H), int(ignore_index), int(piece))


def fbob_linear_ce_workspace_bytes(p: LinearCe, which: int) -> int:
    """Bytes of workspace of the forward (0), backward (1) or its product (2)."""
    return int(load().fbob_linear_ce_workspace_bytes(ctypes.byref(p), which))


def _ce_common(H, W, target, lse=None, g=None):
    index, rows = _device(H, "H"), H.shape[:1]
    _tensor(H, "H", index, H.dtype)
    _tensor(W, "W", index, H.dtype)
    _tensor(target, "target", index, torch.int64, rows)
    _tensor(lse, "lse", index, torch.float32, rows)
    _tensor(g, "g", index, torch.float32, rows)
    return index, rows


def _bytes(p, which, workspace, H, index, stream):
    """(pointer, bytes) of the given uint8 workspace or of a new one."""
    if workspace is None:
        workspace = _new(H, (load().fbob_linear_ce_workspace_bytes(p, which),), torch.uint8, stream)
    else:
        _tensor(workspace, "workspace", index, torch.uint8)
    return workspace.data_ptr(), workspace.numel(), workspace


def fbob_linear_ce_fwd(H, W, target, ignore_index=-100, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse) [T] fp32 of the tokens H [T, D] under logits H W^T, W [V, D];
    target [T] int64.  ``workspace``: uint8."""
    p = linear_ce_for(H, W, ignore_index)
    index, rows = _ce_common(H, W, target)
    loss = _out(loss, "loss", H, index, rows, torch.float32, stream)
    lse = _out(lse, "lse", H, index, rows, torch.float32, stream)
    at, size, workspace = _bytes(p, 0, workspace, H, index, stream)
    _run(load().fbob_linear_ce_fwd, index, stream, p, H.data_ptr(), W.data_ptr(), target.data_ptr(), loss.data_ptr(),
         lse.data_ptr(), at, size)
    return loss, lse


def fbob_linear_ce_bwd(H, W, target, lse, g, ignore_index=-100, piece=0, dH=None, dW=None, want=(True, True),
                       workspace=None, stream=None):
    """(dH, dW) of sum_t g_t loss_t; ``want`` says which to compute.  ``piece``:
    classes whose gradient is held at once (0: chosen by the library)."""
    p = linear_ce_for(H, W, ignore_index, piece)
    index, _ = _ce_common(H, W, target, lse, g)
    dH = _out(dH, "dH", H, index, H.shape, H.dtype, stream) if want[0] else None
    dW = _out(dW, "dW", H, index, W.shape, H.dtype, stream) if want[1] else None
    at, size, workspace = _bytes(p, 1, workspace, H, index, stream)
    _run(load().fbob_linear_ce_bwd, index, stream, p, H.data_ptr(), W.data_ptr(), target.data_ptr(), lse.data_ptr(),
         g.data_ptr(), _p(dH), _p(dW), at, size)
    return dH, dW


def fbob_linear_ce_bob(H, W, target, lse, g, UH, UW, ignore_index=-100, piece=0, gH=None, gW=None, gg=None,
                       want=(True, True, True), workspace=None, stream=None):
    """(gH, gW, gg) = the vector-Jacobian product of (H, W, g) -> (dH, dW)
    along (UH, UW), one of which may be None; ``want`` says which to compute."""
    p = linear_ce_for(H, W, ignore_index, piece)
    index, rows = _ce_common(H, W, target, lse, g)
    _tensor(UH, "UH", index, H.dtype, H.shape)
    _tensor(UW, "UW", index, H.dtype, W.shape)
    gH = _out(gH, "gH", H, index, H.shape, H.dtype, stream) if want[0] else None
    gW = _out(gW, "gW", H, index, W.shape, H.dtype, stream) if want[1] else None
    gg = _out(gg, "gg", H, index, rows, torch.float32, stream) if want[2] else None
    at, size, workspace = _bytes(p, 2, workspace, H, index, stream)
    _run(load().fbob_linear_ce_bob, index, stream, p, H.data_ptr(), W.data_ptr(), target.data_ptr(), lse.data_ptr(),
         g.data_ptr(), _p(UH), _p(UW), _p(gH), _p(gW), _p(gg), at, size)
    return gH, gW, gg
