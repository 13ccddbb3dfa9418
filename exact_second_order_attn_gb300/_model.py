"""ctypes binding of the operators around the attention: argument marshalling
only, like ``_lib`` (include/fbob.h has each call's contract).

The calls run on the device of their tensors, on ``stream`` or that device's
current stream; outputs and workspaces that are not given come from torch's
allocator on that stream.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import LinearCe, Norm, Rotary, RotaryHeads, _check, _ptr, load

DTYPES = {torch.bfloat16: _lib.BF16, torch.float32: _lib.FP32}


def _dtype(t):
    try:
        return DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _tensor(t, name, like, dtype, shape=None):
    """Check one contiguous tensor argument (None passes)."""
    if t is None:
        return
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _run(entry, like, stream, *args):
    """Call a launching entry point with ``like``'s device current."""
    fn = getattr(load(), entry)
    if torch.cuda.current_device() == like.device.index:
        if stream is None:
            stream = torch.cuda.current_stream()
        _check(fn(*args, ctypes.c_void_p(stream.cuda_stream)))
        return
    with torch.cuda.device(like.device):
        if stream is None:
            stream = torch.cuda.current_stream()
        _check(fn(*args, ctypes.c_void_p(stream.cuda_stream)))


def _new(like, shape, dtype, stream):
    """An uninitialised tensor of ``stream``'s pool (memory that other streams
    may still be using is not handed to it)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


# --- rotary positions -----------------------------------------------------------------------------

def fbob_rotary_frequencies(rotary: Rotary) -> list:
    """theta_i of the description, scaled (i < rot/2)."""
    out = (ctypes.c_double * max(1, rotary.rot // 2))()
    _check(load().fbob_rotary_frequencies(ctypes.byref(rotary), out))
    return list(out)


def _heads(t, name, like):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, d]")
    if not t.is_cuda or t.device != like.device:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device")
    if t.dtype != like.dtype:
        raise TypeError(f"{name}: expected {like.dtype}, got {t.dtype}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name}: the columns of a head must be contiguous")


def fbob_rotary_apply(rotary, Q, K=None, positions=None, offset=0, transpose=False, Qo=None, Ko=None, stream=None):
    """Rotary positions on Q [B, H, N, d] and K [B, Hk, N, d] (any strides over
    contiguous rows) in one launch: (Qo, Ko), or Qo alone without K; contiguous
    [B, H, N, d] if not given.  ``positions``: int32 or int64, [N] or [B, N],
    added to ``offset``; without them token n has position offset + n.
    ``transpose``: the map's transpose (gradients)."""
    _heads(Q, "Q", Q)
    dt = _dtype(Q)
    B, H, N, d = Q.shape
    pairs = [("Q", Q, _new(Q, Q.shape, Q.dtype, stream) if Qo is None else Qo)]
    if K is not None:
        _heads(K, "K", Q)
        if K.shape[0] != B or K.shape[2:] != Q.shape[2:]:
            raise ValueError(f"K: expected shape ({B}, Hk, {N}, {d}), got {tuple(K.shape)}")
        pairs.append(("K", K, _new(Q, K.shape, Q.dtype, stream) if Ko is None else Ko))
    elif Ko is not None:
        raise ValueError("Ko without K")
    t = (RotaryHeads * len(pairs))()
    for e, (name, x, y) in zip(t, pairs):
        _heads(y, name + "o", Q)
        if y.shape != x.shape:
            raise ValueError(f"{name}o: expected shape {tuple(x.shape)}, got {tuple(y.shape)}")
        e.x, e.y, e.H = x.data_ptr(), y.data_ptr(), x.shape[1]
        e.x_stride[:], e.y_stride[:] = x.stride()[:3], y.stride()[:3]
    size, step = 0, 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        if not positions.is_cuda or positions.device != Q.device:
            raise ValueError("positions: all tensors must be on the same CUDA device")
        if tuple(positions.shape) not in ((N,), (B, N)):
            raise ValueError(f"positions: expected shape ({N},) or ({B}, {N}), got {tuple(positions.shape)}")
        if N > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous")
        size = positions.element_size()
        step = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    _run("fbob_rotary_apply", Q, stream, ctypes.byref(rotary), B, N, d, dt, t, len(pairs), _ptr(positions), size, step,
         int(offset), int(bool(transpose)))
    return pairs[0][2] if K is None else (pairs[0][2], pairs[1][2])


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


def _norm_workspace(p, x, need, workspace, stream):
    if workspace is None:
        workspace = _new(x, (max(1, need) + 3) // 4, torch.float32, stream)
    _tensor(workspace, "workspace", x, torch.float32)
    return workspace


def fbob_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """(y, mean, rstd) = layer norm over the last dimension of x (contiguous,
    any leading shape); mean and rstd are fp32 of the leading shape."""
    wt = _weight_dtype(x, weight, bias)
    p = norm_for(x, wt, eps)
    _tensor(x, "x", x, x.dtype)
    _tensor(weight, "weight", x, wt, x.shape[-1:])
    _tensor(bias, "bias", x, wt, x.shape[-1:])
    y = _new(x, x.shape, x.dtype, stream) if y is None else y
    mean = _new(x, x.shape[:-1], torch.float32, stream) if mean is None else mean
    rstd = _new(x, x.shape[:-1], torch.float32, stream) if rstd is None else rstd
    _tensor(y, "y", x, x.dtype, x.shape)
    _tensor(mean, "mean", x, torch.float32, x.shape[:-1])
    _tensor(rstd, "rstd", x, torch.float32, x.shape[:-1])
    _run("fbob_layer_norm_fwd", x, stream, ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean),
         _ptr(rstd))
    return y, mean, rstd


def _norm_common(x, weight, mean, rstd, dy):
    _tensor(x, "x", x, x.dtype)
    _tensor(mean, "mean", x, torch.float32, x.shape[:-1])
    _tensor(rstd, "rstd", x, torch.float32, x.shape[:-1])
    _tensor(dy, "dy", x, x.dtype, x.shape)
    if weight is not None:
        _tensor(weight, "weight", x, weight.dtype, x.shape[-1:])


def fbob_layer_norm_bwd(x, weight, mean, rstd, dy, dx=None, dw=None, db=None, want=(True, True, True),
                        bias_dtype=None, workspace=None, stream=None):
    """(dx, dw, db) = layer norm's backward; ``want`` says which to compute
    (the others are None).  dw needs ``weight``; without one db has
    ``bias_dtype`` (default: x's)."""
    wt = weight.dtype if weight is not None else bias_dtype or x.dtype
    p = norm_for(x, wt)
    _norm_common(x, weight, mean, rstd, dy)
    want = (want[0], want[1] and weight is not None, want[2])
    dx = (_new(x, x.shape, x.dtype, stream) if dx is None else dx) if want[0] else None
    dw = (_new(x, x.shape[-1:], wt, stream) if dw is None else dw) if want[1] else None
    db = (_new(x, x.shape[-1:], wt, stream) if db is None else db) if want[2] else None
    _tensor(dx, "dx", x, x.dtype, x.shape)
    _tensor(dw, "dw", x, wt, x.shape[-1:])
    _tensor(db, "db", x, wt, x.shape[-1:])
    need = 0
    if want[1] or want[2]:
        need = fbob_layer_norm_workspace_bytes(p) // (1 if want[1] and want[2] else 2)
    workspace = _norm_workspace(p, x, need, workspace, stream)
    _run("fbob_layer_norm_bwd", x, stream, ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy),
         _ptr(dx), _ptr(dw), _ptr(db), _ptr(workspace), ctypes.c_size_t(workspace.numel() * 4))
    return dx, dw, db


def fbob_layer_norm_bob(x, weight, mean, rstd, dy, ux, uw=None, ub=None, gx=None, gw=None, gdy=None,
                        want=(True, True, True), workspace=None, stream=None):
    """(gx, gw, gdy) = the vector-Jacobian product of layer norm's backward
    along (ux, uw, ub); ``want`` says which to compute.  gw needs ``weight``."""
    wt = _weight_dtype(x, weight, uw, ub)
    p = norm_for(x, wt)
    _norm_common(x, weight, mean, rstd, dy)
    _tensor(ux, "ux", x, x.dtype, x.shape)
    _tensor(uw, "uw", x, wt, x.shape[-1:])
    _tensor(ub, "ub", x, wt, x.shape[-1:])
    want = (want[0], want[1] and weight is not None, want[2])
    gx = (_new(x, x.shape, x.dtype, stream) if gx is None else gx) if want[0] else None
    gw = (_new(x, x.shape[-1:], wt, stream) if gw is None else gw) if want[1] else None
    gdy = (_new(x, x.shape, x.dtype, stream) if gdy is None else gdy) if want[2] else None
    _tensor(gx, "gx", x, x.dtype, x.shape)
    _tensor(gw, "gw", x, wt, x.shape[-1:])
    _tensor(gdy, "gdy", x, x.dtype, x.shape)
    workspace = _norm_workspace(p, x, fbob_layer_norm_workspace_bytes(p) // 2 if want[1] else 0, workspace, stream)
    _run("fbob_layer_norm_bob", x, stream, ctypes.byref(p), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy),
         _ptr(ux), _ptr(uw), _ptr(ub), _ptr(gx), _ptr(gw), _ptr(gdy), _ptr(workspace),
         ctypes.c_size_t(workspace.numel() * 4))
    return gx, gw, gdy


# --- cross entropy of a linear head -----------------------------------------------------------------

def linear_ce_for(H: torch.Tensor, W: torch.Tensor, ignore_index: int = -100, piece: int = 0) -> LinearCe:
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError(f"H [T, D] and W [V, D] are needed, got {tuple(H.shape)} and {tuple(W.shape)}")
    if max(H.shape[0], W.shape[0], W.shape[1]) > 2 ** 31 - 1:
        raise ValueError("sizes must fit 32 bits")
    return LinearCe(H.shape[0], H.shape[1], W.shape[0], _dtype(H), int(ignore_index), int(piece))


def fbob_linear_ce_workspace_bytes(p: LinearCe, which: int) -> int:
    """Bytes of workspace of the forward (0), backward (1) or its product (2)."""
    return int(load().fbob_linear_ce_workspace_bytes(ctypes.byref(p), which))


def _ce_common(H, W, target, lse=None, g=None):
    _tensor(H, "H", H, H.dtype)
    _tensor(W, "W", H, H.dtype)
    _tensor(target, "target", H, torch.int64, H.shape[:1])
    _tensor(lse, "lse", H, torch.float32, H.shape[:1])
    _tensor(g, "g", H, torch.float32, H.shape[:1])


def _ce_workspace(p, which, H, workspace, stream):
    if workspace is None:
        workspace = _new(H, (fbob_linear_ce_workspace_bytes(p, which),), torch.uint8, stream)
    _tensor(workspace, "workspace", H, torch.uint8)
    return workspace, ctypes.c_size_t(workspace.numel())


def fbob_linear_ce_fwd(H, W, target, ignore_index=-100, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse) [T] fp32 of the tokens H [T, D] under logits H W^T, W [V, D];
    target [T] int64.  ``workspace``: uint8."""
    p = linear_ce_for(H, W, ignore_index)
    _ce_common(H, W, target)
    loss = _new(H, H.shape[:1], torch.float32, stream) if loss is None else loss
    lse = _new(H, H.shape[:1], torch.float32, stream) if lse is None else lse
    _tensor(loss, "loss", H, torch.float32, H.shape[:1])
    _tensor(lse, "lse", H, torch.float32, H.shape[:1])
    workspace, size = _ce_workspace(p, 0, H, workspace, stream)
    _run("fbob_linear_ce_fwd", H, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(target), _ptr(loss), _ptr(lse),
         _ptr(workspace), size)
    return loss, lse


def fbob_linear_ce_bwd(H, W, target, lse, g, ignore_index=-100, piece=0, dH=None, dW=None, want=(True, True),
                       workspace=None, stream=None):
    """(dH, dW) of sum_t g_t loss_t; ``want`` says which to compute.  ``piece``:
    classes whose gradient is held at once (0: chosen by the library)."""
    p = linear_ce_for(H, W, ignore_index, piece)
    _ce_common(H, W, target, lse, g)
    dH = (_new(H, H.shape, H.dtype, stream) if dH is None else dH) if want[0] else None
    dW = (_new(H, W.shape, H.dtype, stream) if dW is None else dW) if want[1] else None
    _tensor(dH, "dH", H, H.dtype, H.shape)
    _tensor(dW, "dW", H, H.dtype, W.shape)
    workspace, size = _ce_workspace(p, 1, H, workspace, stream)
    _run("fbob_linear_ce_bwd", H, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(target), _ptr(lse), _ptr(g), _ptr(dH),
         _ptr(dW), _ptr(workspace), size)
    return dH, dW


def fbob_linear_ce_bob(H, W, target, lse, g, UH, UW, ignore_index=-100, piece=0, gH=None, gW=None, gg=None,
                       want=(True, True, True), workspace=None, stream=None):
    """(gH, gW, gg) = the vector-Jacobian product of (H, W, g) -> (dH, dW)
    along (UH, UW), one of which may be None; ``want`` says which to compute."""
    p = linear_ce_for(H, W, ignore_index, piece)
    _ce_common(H, W, target, lse, g)
    _tensor(UH, "UH", H, H.dtype, H.shape)
    _tensor(UW, "UW", H, H.dtype, W.shape)
    gH = (_new(H, H.shape, H.dtype, stream) if gH is None else gH) if want[0] else None
    gW = (_new(H, W.shape, H.dtype, stream) if gW is None else gW) if want[1] else None
    gg = (_new(H, H.shape[:1], torch.float32, stream) if gg is None else gg) if want[2] else None
    _tensor(gH, "gH", H, H.dtype, H.shape)
    _tensor(gW, "gW", H, H.dtype, W.shape)
    _tensor(gg, "gg", H, torch.float32, H.shape[:1])
    workspace, size = _ce_workspace(p, 2, H, workspace, stream)
    _run("fbob_linear_ce_bob", H, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(target), _ptr(lse), _ptr(g), _ptr(UH),
         _ptr(UW), _ptr(gH), _ptr(gW), _ptr(gg), _ptr(workspace), size)
    return gH, gW, gg
