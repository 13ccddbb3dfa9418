"""The linear head's gradients where their sums are cut into chains: over more
than 16,384 tokens or classes, half of that in the second order."""

import pytest
import torch

from test_gpu_linear_ce import chain, compare, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V", [(8192, 40), (8200, 40), (12001, 33), (16384, 24), (16400, 24), (33000, 17), (40, 8200),
                                 (40, 16384), (20, 16390), (20, 33000)])
def test_long_sums(T, V):
    t = make(T, 16, V, "bf16", seed=T + V, ignored=(3,))
    compare(t, chain(t))


def test_long_sums_of_one_sign():
    """Every term of dW has the sign of the result, so that roundings towards
    zero would add up."""
    t = make(20000, 24, 12, "bf16", seed=1)
    for k in ("H", "UH", "g"):
        t[k] = t[k].abs()
    compare(t, chain(t))


def test_long_sums_in_pieces():
    t = make(9000, 16, 600, "bf16", seed=2)
    whole, cut = chain(t), chain(t, piece=256)
    compare(t, cut)
    assert torch.equal(whole["gW"], cut["gW"])
