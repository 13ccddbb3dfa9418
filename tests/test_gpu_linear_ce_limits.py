"""The linear head's cross entropy at the largest sizes that the header allows,
against 64-bit torch operations."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from test_gpu_linear_ce import chain, compare, make

pytestmark = pytest.mark.gpu


def exact(t):
    H, W, UH, UW, g = (t[k].double() for k in ("H", "W", "UH", "UW", "g"))
    y, i = t["target"], torch.arange(len(g), device="cuda")
    z = H @ W.T
    lse = torch.logsumexp(z, -1)
    p = (z - lse[:, None]).exp()
    b = UH @ W.T + H @ UW.T
    alpha = (p * b).sum(-1)
    Z = g[:, None] * p * (b - alpha[:, None])
    G = p * g[:, None]
    G[i, y] -= g
    return dict(loss=lse - z[i, y], dH=G @ W, dW=G.T @ H, gH=Z @ W + G @ UW, gW=Z.T @ H + G.T @ UH, gg=alpha - b[i, y])


@pytest.mark.parametrize("T,D,V", [(3, 4, 1 << 24), (1 << 24, 8, 3)])
def test_most_classes_and_most_tokens(T, D, V):
    """Norms of differences.  Gradients: entries of G and Z and the results are
    rounded to bf16, 2^-8 at most each, which norms do not exceed as the roundings
    are independent: 2^-7.  Losses and gg, fp32 logits of a few columns: 16 roundings
    of 2^-24, times their condition of order ten."""
    t = make(T, D, V, "bf16", seed=2)
    got, ref = chain(t), exact(t)
    for k, r in ref.items():
        off = float((got[k].double() - r).norm() / r.norm())
        assert off <= (2 ** -7 if k in ("dH", "dW", "gH", "gW") else 1e-5), k
    fb.device_status()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_most_columns(dtype):
    t = make(20, 1 << 15, 150, dtype, seed=3, ignored=(2,))
    compare(t, chain(t))
