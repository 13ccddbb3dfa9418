"""Dropout on the GPU against the generator in plain Python."""

import numpy as np
import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from model_helpers import check, draw, misaligned, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (2, 8), (5, 64), (33, 100), (7, 1537), (300, 24)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.9, 1.0])
def test_dropout_against_the_generator(T, D, dtype, p):
    """A product, a sum and the result's rounding."""
    x, r = draw(T, (T, D), dtype), draw(D, (T, D), dtype)
    d = fb.Dropout(p, seed=77 + 2 ** 40, offset=2 ** 64 - 5)
    m = om.dropout_factor(T, D, p, 77 + 2 ** 40, 2 ** 64 - 5)
    X, R = np64(x), np64(r)
    check("y", fb.fbob_dropout_apply(d, x), m * X, np.abs(m * X), 2)
    check("y + r", fb.fbob_dropout_apply(d, x, r), m * X + R, np.abs(m * X) + np.abs(R), 3)
    for a in (misaligned(x),):
        assert torch.equal(fb.fbob_dropout_apply(d, a, r), fb.fbob_dropout_apply(d, x, r))


def test_the_counter_moves_the_offset_modulo_2_64():
    x = draw(1, (9, 40))
    counter = torch.tensor([7], device="cuda")
    a = fb.fbob_dropout_apply(fb.Dropout(0.5, 3, 2 ** 64 - 4), x, counter=counter)
    b = fb.fbob_dropout_apply(fb.Dropout(0.5, 3, 3), x)
    assert torch.equal(a, b)
    counter.fill_(-2)
    assert torch.equal(fb.fbob_dropout_apply(fb.Dropout(0.5, 3, 5), x, counter=counter), b)


def test_leading_dimensions_outputs_and_empty():
    x = draw(2, (2, 3, 5, 24), "bf16")
    d = fb.Dropout(0.4, 1)
    y = torch.full((720 + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    fb.fbob_dropout_apply(d, x, y=y[:720].view(x.shape))
    assert torch.equal(y[:720].view(30, 24), fb.fbob_dropout_apply(d, x.view(30, 24))) and (y[720:] == 9).all()
    assert fb.fbob_dropout_apply(d, x[:0]).shape == (0, 3, 5, 24)
    assert torch.equal(fb.fbob_dropout_apply(d, x[0, 0, 0]), fb.fbob_dropout_apply(d, x.view(30, 24))[0])


def test_more_than_2_31_elements():
    """The first and the last rows of a matrix of 2^31 + 2^20 elements, against
    the generator's words there."""
    D = 4096
    T = 2 ** 19 + 256
    x = torch.ones(T, D, dtype=torch.bfloat16, device="cuda")
    y = fb.fbob_dropout_apply(fb.Dropout(0.5, 5, 6), x)
    for row in (0, 1, T - 1):
        m = [(om.philox([g, row, 6, 0], [5, 0])[j // 2] >> 16 * (j % 2)) % 65536 >= 32768
             for g in range(D // 8) for j in range(8)]
        assert torch.equal(y[row].cpu(), 2.0 * torch.tensor(m).to(torch.bfloat16))


def test_gradients_of_any_order():
    """dx = m g: the map is linear, so a second derivative is the map again."""
    d = fb.Dropout(0.3, 8)
    x, r, g = (draw(i, (6, 20)).requires_grad_() for i in (3, 4, 5))
    y = fb.dropout(d, x, r)
    d.p = 0.9  # the backward draws as its forward did
    dx, dr = torch.autograd.grad(y, (x, r), g, create_graph=True)
    d.p = 0.3
    assert torch.equal(dx, fb.fbob_dropout_apply(d, g.detach())) and torch.equal(dr, g)
    u = draw(6, (6, 20))
    (gg,) = torch.autograd.grad(dx, g, u, create_graph=True)
    assert torch.equal(gg, fb.fbob_dropout_apply(d, u))
    assert not fb.dropout(d, x.detach(), r).grad_fn is None
