"""Calls of the operators' autograd functions that a training program makes
between a forward and its backward."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import U32, draw, misaligned

pytestmark = pytest.mark.gpu


def test_a_rotary_description_changed_after_the_forward():
    """The backward, and its own, turn by the description of their forward."""
    r = fb.Rotary(16, base=10000.0)
    Q = draw(1, (1, 2, 30, 16)).requires_grad_()
    g = draw(2, (1, 2, 30, 16)).requires_grad_()
    want = fb.fbob_rotary_apply(r, g.detach(), transpose=True)
    back = fb.fbob_rotary_apply(r, Q.detach())
    q = fb.rotary(r, Q)
    r.base, r.magnitude, r.interleaved = 500.0, 2.0, 1
    (dQ,) = torch.autograd.grad(q, Q, g, create_graph=True)
    assert torch.equal(dQ, want)
    r.scaling, r.factor = 1, 4.0
    (u,) = torch.autograd.grad(dQ, g, Q.detach())
    assert torch.equal(u, back)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cotangents_that_are_views_of_one_vector(dtype):
    """Parameters and directions cut out of one flat vector start on any element.
    Layer norm then sums in another order: a step of the result's type, and 600
    roundings of magnitudes up to ten times the largest result."""
    T, D, V = 20, 64, 130
    H, W = draw(3, (T, D), dtype), draw(4, (V, D), dtype, 0.2)
    x, w, b = draw(5, (T, D), dtype), draw(6, (D,), dtype, 0.2, 1.0), draw(7, (D,), dtype, 0.2)
    Q = draw(8, (1, 2, 10, 32), dtype)
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(9)).cuda()

    def run(cut):
        ps = [(misaligned(t) if cut else t.clone()).requires_grad_() for t in (H, W, x, w, b, Q)]
        g = draw(10, Q.shape, dtype).requires_grad_()
        outs = (fb.linear_cross_entropy(ps[0], ps[1], y).mean(), (fb.layer_norm(*ps[2:5]) * 2).sin().sum())
        first = torch.autograd.grad(sum(outs), ps[:5], create_graph=True)
        first += torch.autograd.grad(fb.rotary(fb.Rotary(32), ps[5]), ps[5], g, create_graph=True)
        sizes = [t.numel() for t in first]
        flat = draw(11, (sum(sizes) + 1,), dtype)[1:]
        us = [u.view(t.shape) for u, t in zip(flat.split(sizes), first)]
        if not cut:
            us = [u.clone() for u in us]
        return torch.autograd.grad(first, (*ps[:5], g), us)

    for got, ref in zip(run(True), run(False)):
        off, ref = (got.double() - ref.double()).abs(), ref.double().abs()
        assert (off <= torch.finfo(dtype).eps * ref + 6000 * U32 * ref.max()).all()
    fb.device_status()
