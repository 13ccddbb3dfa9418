"""Activations and slopes of linear layers element by element, where no sum hides them."""

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


def reference(act, z):
    """(a, a', a'', size of the exponent) in 64 bits, without cancellation where they are small."""
    if act == "gelu":
        from scipy.special import ndtr
        f = np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        return z * ndtr(z), ndtr(z) + z * f, f * (2 - z * z), z * z
    k = 2 * np.sqrt(2 / np.pi)
    v, v1, v2 = (z, 1.0, 0.0) if act == "silu" else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z * z), k * 0.26829 * z)
    e = np.exp(-np.abs(v))
    s, d, w = np.where(v >= 0, 1, e) / (1 + e), e / (1 + e) ** 2, np.where(v >= 0, -1, 1) * (1 - e) / (1 + e)
    return z * s, s + z * d * v1, d * (2 * v1 + z * v2 + z * v1 * v1 * w), np.abs(v)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_and_slopes_by_element(dtype, few, act):
    """Layers of one column whose products are z, a, a' and a'' themselves (few: one
    token and an output for each z; else a token for each).

    Over all z: within 2^-18 (bf16) or 2^-21 (fp32) of 1 + |z|, and the roundings of the
    results (and of q, once with more than 16 tokens).  In the tails (a and a' at z <= -3, a''
    at |z| >= 3) relative to the values: the exponent, of size v, is off by a few roundings of
    its terms, which the exponential turns into as many times v relative ones; beside them the
    functions take some twenty roundings in fp32, and 2^-12 of the normal integral in bf16
    (2^-11 with the exponent's part, v up to 90)."""
    z = torch.linspace(-10, 10, 4001).to(TYPES[dtype])
    n, one = len(z), torch.ones(1, 1, dtype=z.dtype, device="cuda")
    col, ones = z.view(n, 1).cuda(), torch.ones(n, 1, dtype=z.dtype, device="cuda")
    if few:  # z = x W^T, t = x uW^T = 1, gW = q
        y, kept = fb.fbob_linear_fwd(one, col, activation=act)
        _, gW, _, gdy = fb.fbob_linear_bob(one, col, kept, ones.T.contiguous(), None, ones, None, act)
        a2 = gW
    else:    # t = ux W^T = 1, gx = q
        y, kept = fb.fbob_linear_fwd(col, one, activation=act)
        gx, _, _, gdy = fb.fbob_linear_bob(col, one, kept, ones, ones, None, None, act)
        a2 = gx
    fb.device_status()
    z = z.double().numpy()
    bf = dtype == "bf16"
    h = torch.finfo(TYPES[dtype]).eps / 2
    once = h * (2 + h) if bf and not few else h * (1 + 2 ** -6)  # roundings of a''
    near = 2.0 ** (-18 if bf else -21) * (1 + np.abs(z))
    *refs, v = reference(act, z)
    rel = 2.0 ** -11 if bf else 2.0 ** -24 * (32 + 8 * v)
    for name, got, ref, r, tail in (("a", y, refs[0], h, z <= -3), ("a'", gdy, refs[1], h, z <= -3),
                                    ("a''", a2, refs[2], once, np.abs(z) >= 3)):
        off = np.abs(np64(got).reshape(-1) - ref)
        assert (off <= r * np.abs(ref) + (1 + r) * near).all(), (name, z[np.argmax(off - r * np.abs(ref) - near)])
        far = off > (r + (1 + r) * rel) * np.abs(ref)
        assert not (far & tail).any(), (name, z[far & tail], (off / np.abs(ref))[far & tail])
