"""Slopes of linear layers where z is as small as its type allows."""

import numpy as np
import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import TYPES, check, draw, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K", [(6, 8), (40, 8), (300, 24), (40, 2056)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_relu_slopes_of_small_z(dtype, T, K):
    """z is one exact product of magnitudes from 2^-110 on (K = 2056: summed in slabs):
    slopes are 1 where z > 0, as small as it may be."""
    N = 40
    t = dict(x=torch.zeros(T, K), W=draw(1, (N, K), device="cpu"), dy=draw(2, (T, N), device="cpu"),
             ux=draw(3, (T, K), device="cpu"), uW=draw(4, (N, K), device="cpu"))
    t["x"][:, 0] = draw(5, (T,), device="cpu").sign() * 2.0 ** -torch.arange(T).remainder(61)
    t["W"][:, 0] = draw(6, (N,), device="cpu").sign() * 2.0 ** -torch.arange(N).mul(7).remainder(51)
    t = {k: v.to(TYPES[dtype]).cuda() for k, v in t.items()}
    y, z = fb.fbob_linear_fwd(t["x"], t["W"], activation="relu")
    dx, dW, db = fb.fbob_linear_bwd(t["x"], t["W"], z, t["dy"], "relu")
    gx, gW, gb, gdy = fb.fbob_linear_bob(t["x"], t["W"], z, t["dy"], t["ux"], t["uW"], None, "relu")
    fb.device_status()
    x, W, dy, ux, uW = (np64(t[k]) for k in ("x", "W", "dy", "ux", "uW"))
    Z = x @ W.T
    up = Z > 0
    assert (np64(y) == Z * up).all() and ((np64(z) > 0) == up).all()
    # (dz is dy or 0: not rounded again)
    dz, s = dy * up, N / 8 + 64
    check("dx", dx, dz @ W, np.abs(dz) @ np.abs(W), s)
    check("dW", dW, dz.T @ x, np.abs(dz).T @ np.abs(x), T / 8 + 64)
    check("db", db, dz.sum(0), np.abs(dz).sum(0), T / 8 + 64)
    tt = np.abs(ux) @ np.abs(W).T + np.abs(x) @ np.abs(uW).T
    check("gdy", gdy, (ux @ W.T + x @ uW.T) * up, tt * up, K / 4 + 64)
    check("gx", gx, dz @ uW, np.abs(dz) @ np.abs(uW), s)
    check("gW", gW, dz.T @ ux, np.abs(dz).T @ np.abs(ux), T / 8 + 64)
    assert not gb.any()
