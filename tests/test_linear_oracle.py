"""The oracle of linear layers and dropout, pinned to torch's fp64 autograd
(first and second order) and to the generator's published answers."""

import numpy as np
import pytest
import torch

import oracle.model as om

ACTS = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
        "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"), "silu": torch.nn.functional.silu}


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], "d16cfe09 94fdcceb 5001e420 24126ea1"),
])
def test_the_generator_gives_its_published_answers(counter, key, words):
    assert om.philox(counter, key) == [int(w, 16) for w in words.split()]


def test_the_mask_has_its_share_and_its_scale():
    """4096 elements of probability 1/4: five standard deviations are 139."""
    m = om.dropout_factor(64, 64, 0.25, 7, 2 ** 40)
    assert set(np.unique(m)) == {0.0, 4 / 3} and abs((m == 0).sum() - 1024) <= 139
    assert (om.dropout_factor(3, 5, 0.0, 7, 0) == 1).all() and (om.dropout_factor(3, 5, 1.0, 7, 0) == 0).all()


@pytest.mark.parametrize("kind", list(ACTS))
def test_linear_matches_autograd(kind):
    g = torch.Generator().manual_seed(3)
    x, W, b, r, dy, ux, uW, ub = (torch.randn(s, generator=g, dtype=torch.float64)
                                  for s in ((5, 7), (9, 7), 9, (5, 9), (5, 9), (5, 7), (9, 7), 9))
    m = om.dropout_factor(5, 9, 0.3, 11, 13)
    leaves = [t.requires_grad_() for t in (x, W, b, dy)]
    y = ACTS[kind](x @ W.T + b) * torch.from_numpy(m) + r
    first = torch.autograd.grad(y, leaves[:3], dy, create_graph=True)
    second = torch.autograd.grad(first, leaves, (ux, uW, ub), allow_unused=True)
    second = [torch.zeros_like(l) if t is None else t for t, l in zip(second, leaves)]
    n = [t.detach().numpy() for t in (x, W, b, r, dy, ux, uW, ub)]
    x, W, b, r, dy, ux, uW, ub = n
    for got, ref in ((om.linear(x, W, b, r, kind, m), y), *zip(om.linear_bwd(x, W, b, dy, kind, m), first),
                     *zip(om.linear_bob(x, W, b, dy, ux, uW, ub, kind, m), second)):
        np.testing.assert_allclose(got, ref.detach().numpy(), rtol=0, atol=1e-12 * 50)
