"""Binding of the operators around the attention: signatures and
documentation; the arguments are checked and marshalled by ``_fbob_model``
(``bind/``), which calls the C ABI (include/fbob.h has each call's contract).

The calls run on the device of their tensors, on ``stream`` or that device's
current stream; outputs and workspaces that are not given come from torch's
allocator on that stream.
"""

from __future__ import annotations

import ctypes
import importlib

import torch

from . import _lib
from ._lib import LinearCe, Norm, Rotary, _check, load

DTYPES = {torch.bfloat16: _lib.BF16, torch.float32: _lib.FP32}

_ext = None


def _bind():
    """The compiled binding (raises if it has not been built)."""
    global _ext
    if _ext is None:
        load()
        try:
            ext = importlib.import_module("._fbob_model", __package__)
        except ImportError as e:
            raise RuntimeError("the binding of the model operators is missing: build it with "
                               "exact_second_order_attn_gb300.build.build()") from e
        ext.set_check(_check)
        _ext = ext
    return _ext


def _call(name, stream, *args):
    """Call the binding; on another stream than the current one with that
    stream (and its device) current, so that what it allocates is that
    stream's."""
    f = getattr(_ext or _bind(), name)
    if stream is None:
        return f(*args)
    for a in args:
        if isinstance(a, torch.Tensor):  # the binding holds the others to the first one's device
            if stream.device != a.device:
                raise ValueError(f"stream: of {stream.device}, the tensors are on {a.device}")
            break
    with torch.cuda.stream(stream):
        return f(*args)


def _code(dtype):
    try:
        return DTYPES[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None


# --- rotary positions -----------------------------------------------------------------------------

def fbob_rotary_frequencies(rotary: Rotary) -> list:
    """theta_i of the description, scaled (i < rot/2)."""
    out = (ctypes.c_double * max(1, rotary.rot // 2))()
    _check(load().fbob_rotary_frequencies(ctypes.byref(rotary), out))
    return list(out)


def fbob_rotary_apply(rotary, Q, K=None, positions=None, offset=0, transpose=False, Qo=None, Ko=None, stream=None):
    """Rotary positions on Q [B, H, N, d] and K [B, Hk, N, d] (any strides over
    contiguous rows) in one launch: (Qo, Ko), or Qo alone without K; contiguous
    [B, H, N, d] if not given.  ``positions``: int32 or int64, [N] or [B, N],
    added to ``offset``; without them token n has position offset + n.
    ``transpose``: the map's transpose (gradients)."""
    return _call("rotary_apply", stream, rotary, Q, K, positions, offset, transpose, Qo, Ko)


# --- layer norm -----------------------------------------------------------------------------------

def norm_for(x: torch.Tensor, weight_dtype: torch.dtype, eps: float = 0.0) -> Norm:
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    D = x.shape[-1]
    return Norm(x.numel() // D if D else 0, D, _code(x.dtype), _code(weight_dtype), float(eps))


def fbob_layer_norm_workspace_bytes(p: Norm) -> int:
    return int(load().fbob_layer_norm_workspace_bytes(ctypes.byref(p)))


def fbob_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None, stream=None):
    """(y, mean, rstd) = layer norm over the last dimension of x (contiguous,
    any leading shape); mean and rstd are fp32 of the leading shape."""
    return _call("layer_norm_fwd", stream, x, weight, bias, eps, y, mean, rstd)


def fbob_layer_norm_bwd(x, weight, mean, rstd, dy, dx=None, dw=None, db=None, want=(True, True, True),
                        bias_dtype=None, workspace=None, stream=None):
    """(dx, dw, db) = layer norm's backward; ``want`` says which to compute
    (the others are None).  dw needs ``weight``; without one db has
    ``bias_dtype`` (default: x's)."""
    return _call("layer_norm_bwd", stream, x, weight, mean, rstd, dy, dx, dw, db, *want,
                 None if bias_dtype is None else _code(bias_dtype), workspace)


def fbob_layer_norm_bob(x, weight, mean, rstd, dy, ux, uw=None, ub=None, gx=None, gw=None, gdy=None,
                        want=(True, True, True), workspace=None, stream=None):
    """(gx, gw, gdy) = the vector-Jacobian product of layer norm's backward
    along (ux, uw, ub); ``want`` says which to compute.  gw needs ``weight``."""
    return _call("layer_norm_bob", stream, x, weight, mean, rstd, dy, ux, uw, ub, gx, gw, gdy, *want, workspace)


# --- cross entropy of a linear head -----------------------------------------------------------------

def linear_ce_for(H: torch.Tensor, W: torch.Tensor, ignore_index: int = -100, piece: int = 0) -> LinearCe:
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError(f"H [T, D] and W [V, D] are needed, got {tuple(H.shape)} and {tuple(W.shape)}")
    (T, D), V = H.shape, W.shape[0]
    if max(T, D, V) > 2 ** 31 - 1:
        raise ValueError("sizes must fit 32 bits")
    return LinearCe(T, D, V, _code(H.dtype), int(ignore_index), int(piece))


def fbob_linear_ce_workspace_bytes(p: LinearCe, which: int) -> int:
    """Bytes of workspace of the forward (0), backward (1) or its product (2)."""
    return int(load().fbob_linear_ce_workspace_bytes(ctypes.byref(p), which))


def fbob_linear_ce_fwd(H, W, target, ignore_index=-100, loss=None, lse=None, workspace=None, stream=None):
    """(loss, lse) [T] fp32 of the tokens H [T, D] under logits H W^T, W [V, D];
    target [T] int64.  ``workspace``: uint8."""
    return _call("linear_ce_fwd", stream, H, W, target, ignore_index, loss, lse, workspace)


def fbob_linear_ce_bwd(H, W, target, lse, g, ignore_index=-100, piece=0, dH=None, dW=None, want=(True, True),
                       workspace=None, stream=None):
    """(dH, dW) of sum_t g_t loss_t; ``want`` says which to compute.  ``piece``:
    classes whose gradient is held at once (0: chosen by the library)."""
    return _call("linear_ce_bwd", stream, H, W, target, lse, g, ignore_index, piece, dH, dW, *want, workspace)


def fbob_linear_ce_bob(H, W, target, lse, g, UH, UW, ignore_index=-100, piece=0, gH=None, gW=None, gg=None,
                       want=(True, True, True), workspace=None, stream=None):
    """(gH, gW, gg) = the vector-Jacobian product of (H, W, g) -> (dH, dW)
    along (UH, UW), one of which may be None; ``want`` says which to compute."""
    return _call("linear_ce_bob", stream, H, W, target, lse, g, UH, UW, ignore_index, piece, gH, gW, gg, *want, workspace)
