"""PyTorch autograd integration of the operators around the attention.

``rotary``, ``layer_norm``, ``linear``, ``dropout`` and ``linear_cross_entropy`` can be differentiated
twice, like ``attention``, so that ``hvp`` passes through a model built of them.  Outputs and gradients
have the inputs' dtypes; sums and statistics are fp32 inside the kernels.
Third derivatives are not provided (rotary and dropout, linear maps, have all of them).

Every computation runs in the library; this module only moves tensors between
autograd and the binding.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _model
from ._lib import Dropout, Rotary


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
    """A head (or another operand of a product, or its cotangent) where the kernels
    read it in place: bf16 rows of whole 16 bytes have to start on 16 (a view of a
    flat vector need not)."""
    off = (w is not None and w.dtype == torch.bfloat16 and w.dim() >= 1 and w.shape[-1] % 8 == 0
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


def _description(d):
    """A copy of a ``Dropout``, which a later change of ``d`` does not reach."""
    if not isinstance(d, Dropout):
        raise TypeError("dropout: a Dropout description is needed")
    return Dropout.from_buffer_copy(d)


class _Dropout(torch.autograd.Function):
    """(x, residual) -> residual + m x; the backward is the same map of x."""

    @staticmethod
    def forward(ctx, x, residual, counter, d):
        ctx.save_for_backward(counter)
        ctx.d = d
        return _model.fbob_dropout_apply(d, x, residual, counter)

    @staticmethod
    def backward(ctx, g):
        (counter,) = ctx.saved_tensors
        dx = _Dropout.apply(g.contiguous(), None, counter, ctx.d) if ctx.needs_input_grad[0] else None
        return dx, (g if ctx.needs_input_grad[1] else None), None, None


def dropout(d, x, residual=None, counter=None):
    """residual + m x with the mask m that ``d`` (a ``Dropout``) describes, which
    is drawn again for the gradients and never stored.  The last dimension of the
    contiguous x holds the mask's columns.  ``counter``: one int64 element on the
    device, added to the offset when the call runs; gradients read it again, so
    it has to stay until they have run."""
    if not x.is_contiguous() or not (residual is None or residual.is_contiguous()):
        raise ValueError("x and residual must be contiguous")
    # the backward draws by the description as it is now, whatever becomes of d
    return _Dropout.apply(x, residual, counter, _description(d))


class _LinearBwd(torch.autograd.Function):
    """(x, W, bias, dy) -> (dx, dW, db); its own backward is fbob_linear_bob."""

    @staticmethod
    def forward(ctx, x, W, bias, dy, z, counter, how, want):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, W, dy, z, counter)
        ctx.how = how
        return _model.fbob_linear_bwd(_head(x), _head(W), z, _head(dy), *how, counter, want=want)

    @staticmethod
    @once_differentiable
    def backward(ctx, ux, uW, ub):
        x, W, dy, z, counter = ctx.saved_tensors
        want = ctx.needs_input_grad[:4]
        if (ux is None and uW is None and ub is None) or not any(want):
            return None, None, None, None, None, None, None, None
        if ux is None and uW is None:
            ux = torch.zeros_like(x)
        ux, uW, ub = (None if u is None else _head(u.contiguous()) for u in (ux, uW, ub))
        gx, gW, gb, gdy = _model.fbob_linear_bob(_head(x), _head(W), z, _head(dy), ux, uW, ub, *ctx.how, counter,
                                                 want=want)
        return gx, gW, gb, gdy, None, None, None, None


class _Linear(torch.autograd.Function):
    """(x, W, bias, residual) -> y; its backward is the differentiable _LinearBwd."""

    @staticmethod
    def forward(ctx, x, W, bias, residual, counter, how, keep):
        y, z = _model.fbob_linear_fwd(_head(x), _head(W), bias, residual, *how, counter, keep=keep)
        ctx.save_for_backward(x, W, bias, z, counter)
        ctx.how = how
        return y

    @staticmethod
    def backward(ctx, gy):
        x, W, bias, z, counter = ctx.saved_tensors
        want = ctx.needs_input_grad[:3]
        dx = dW = db = None
        if any(want):
            dx, dW, db = _LinearBwd.apply(x, W, bias, gy.contiguous(), z, counter, ctx.how, want)
        return dx, dW, db, (gy if ctx.needs_input_grad[3] else None), None, None, None


def linear(x, weight, bias=None, residual=None, activation="none", dropout=None, counter=None):
    """residual + m a(x weight^T + bias) of a contiguous x [..., K] and weight
    [N, K], twice differentiable; bias [N], residual [..., N], the activation
    ("relu", "gelu", "gelu_tanh", "silu") and the ``Dropout`` m (with its
    ``counter``, as for ``dropout``) are optional.  All tensors have x's dtype."""
    if not all(t is None or t.is_contiguous() for t in (x, weight, bias, residual)):
        raise ValueError("x, weight, bias and residual must be contiguous")
    keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias))
    how = activation, None if dropout is None else _description(dropout)
    return _Linear.apply(x, weight, bias, residual, counter, how, keep)
