"""PyTorch autograd integration of the operators around the attention.

``rotary``, ``layer_norm`` and ``linear_cross_entropy`` can be differentiated
twice, like ``attention``, so that ``hvp`` passes through a model built of them.  Outputs and gradients
have the inputs' dtypes; sums and statistics are fp32 inside the kernels.
Third derivatives are not provided (rotary, a linear map, has all of them).

Every computation runs in the library; this module only moves tensors between
autograd and the binding.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _model
from ._lib import Rotary


def _rows(t):
    """A gradient with contiguous head rows (autograd may hand over any view)."""
    return t if t is None or t.shape[3] <= 1 or t.stride(3) == 1 else t.contiguous()


class _Rotary(torch.autograd.Function):
    """(Q, K) -> the rotated (Q, K); the backward is the transposed map."""

    @staticmethod
    def forward(ctx, Q, K, positions, rotary, offset, transpose):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.args = rotary, offset, transpose
        if Q is None:
            return None, _model.fbob_rotary_apply(rotary, K, None, positions, offset, transpose)
        if K is None:
            return _model.fbob_rotary_apply(rotary, Q, None, positions, offset, transpose), None
        return _model.fbob_rotary_apply(rotary, Q, K, positions, offset, transpose)

    @staticmethod
    def backward(ctx, gQ, gK):
        (positions,) = ctx.saved_tensors
        rotary, offset, transpose = ctx.args
        gQ = _rows(gQ) if ctx.needs_input_grad[0] else None
        gK = _rows(gK) if ctx.needs_input_grad[1] else None
        if gQ is None and gK is None:
            return None, None, None, None, None, None
        dQ, dK = _Rotary.apply(gQ, gK, positions, rotary, offset, not transpose)
        return dQ, dK, None, None, None, None


def rotary(r, Q, K=None, positions=None, offset=0):
    """Rotary positions on Q [B, H, N, d] and K [B, Hk, N, d] as ``r`` (a
    ``Rotary``) describes them, in one launch: (Q', K'), or Q' alone without K.
    Q and K may be strided views with contiguous rows (of a packed projection,
    say); the results are contiguous, as ``attention`` takes them.
    ``positions``: int32 or int64, [N] or [B, N], added to ``offset``; without
    them token n has position offset + n."""
    # the backward turns by the description as it is now, whatever becomes of r
    out = _Rotary.apply(Q, K, positions, Rotary.from_buffer_copy(r), int(offset), False)
    return out[0] if K is None else out


class _NormBwd(torch.autograd.Function):
    """(x, w, dy) -> (dx, dw, db); its own backward is fbob_layer_norm_bob."""

    @staticmethod
    def forward(ctx, x, w, dy, mean, rstd, want, bias_dtype):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, w, dy, mean, rstd)
        return _model.fbob_layer_norm_bwd(x, w, mean, rstd, dy, want=want, bias_dtype=bias_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, ux, uw, ub):
        x, w, dy, mean, rstd = ctx.saved_tensors
        want = ctx.needs_input_grad[:3]
        if (ux is None and uw is None and ub is None) or not any(want):
            return None, None, None, None, None, None, None
        wt = next((u.dtype for u in (w, uw, ub) if u is not None), x.dtype)
        ux = torch.zeros_like(x) if ux is None else ux.contiguous()
        uw, ub = (None if u is None else u.to(wt).contiguous() for u in (uw, ub))
        gx, gw, gdy = _model.fbob_layer_norm_bob(x, w, mean, rstd, dy, ux, uw, ub, want=want)
        return gx, gw, gdy, None, None, None, None


class _Norm(torch.autograd.Function):
    """(x, w, b) -> y; its backward is the differentiable _NormBwd."""

    @staticmethod
    def forward(ctx, x, w, b, eps):
        y, mean, rstd = _model.fbob_layer_norm_fwd(x, w, b, eps)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.bias_dtype = None if b is None else b.dtype
        return y

    @staticmethod
    def backward(ctx, gy):
        x, w, mean, rstd = ctx.saved_tensors
        dx, dw, db = _NormBwd.apply(x, w, gy.contiguous(), mean, rstd, ctx.needs_input_grad[:3], ctx.bias_dtype)
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension of a contiguous x, twice
    differentiable; weight and bias are optional (fp32, or bf16 with a bf16
    x)."""
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    return _Norm.apply(x, weight, bias, float(eps))


def _head(w):
    """A head (or its cotangent) where the kernels read it in place: bf16 rows
    of whole 16 bytes have to start on 16 (a view of a flat vector need not)."""
    off = (w is not None and w.dtype == torch.bfloat16 and w.dim() == 2 and w.shape[1] % 8 == 0
           and w.data_ptr() % 16 != 0)
    return w.clone() if off else w


class _CeBwd(torch.autograd.Function):
    """(H, W, g) -> (dH, dW); its own backward is fbob_linear_ce_bob."""

    @staticmethod
    def forward(ctx, H, W, g, target, lse, ignore_index, want):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(H, W, g, target, lse)
        ctx.ignore_index = ignore_index
        return _model.fbob_linear_ce_bwd(H, _head(W), target, lse, g, ignore_index, want=want)

    @staticmethod
    @once_differentiable
    def backward(ctx, UH, UW):
        H, W, g, target, lse = ctx.saved_tensors
        want = ctx.needs_input_grad[:3]
        if (UH is None and UW is None) or not any(want):
            return None, None, None, None, None, None, None
        UH, UW = (None if u is None else u.contiguous() for u in (UH, UW))
        gH, gW, gg = _model.fbob_linear_ce_bob(H, _head(W), target, lse, g, UH, _head(UW), ctx.ignore_index, want=want)
        return gH, gW, gg, None, None, None, None


class _Ce(torch.autograd.Function):
    """(H, W) -> loss per token; its backward is the differentiable _CeBwd."""

    @staticmethod
    def forward(ctx, H, W, target, ignore_index):
        loss, lse = _model.fbob_linear_ce_fwd(H, _head(W), target, ignore_index)
        ctx.save_for_backward(H, W, target, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    def backward(ctx, g):
        H, W, target, lse = ctx.saved_tensors
        dH, dW = _CeBwd.apply(H, W, g.contiguous(), target, lse, ctx.ignore_index, ctx.needs_input_grad[:2])
        return dH, dW, None, None


def linear_cross_entropy(H, W, target, ignore_index=-100):
    """Losses [T] (fp32) of tokens H [T, D] under the logits H W^T of a head
    W [V, D], twice differentiable in H and W; 0 where target [T] (int64) is
    ``ignore_index``.  The logits are never stored.  A target outside [0, V)
    that is not ``ignore_index`` gives a NaN loss and no gradient, and
    ``device_status`` reports it."""
    if not (H.is_contiguous() and W.is_contiguous() and target.is_contiguous()):
        raise ValueError("H, W and target must be contiguous")
    return _Ce.apply(H, W, target, int(ignore_index))
