"""Calls of the operators' autograd functions that a training program makes
between a forward and its backward."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import draw

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
