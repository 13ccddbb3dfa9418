"""The oracle of the operators around the attention, pinned to torch's fp64
autograd (first and second order), to closed forms and to differences."""

import math

import numpy as np
import pytest
import torch

import oracle.model as om

TOL = 1e-10  # fp64, a few hundred terms per sum


def close(a, b, tol=TOL):
    a, b = np.asarray(a), np.asarray(b.detach() if torch.is_tensor(b) else b)
    scale = max(1.0, np.abs(b).max()) if b.size else 1.0
    assert a.shape == b.shape and (not a.size or np.abs(a - b).max() <= tol * scale)


def randn(seed, *shapes):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g, dtype=torch.float64) for s in shapes]


@pytest.mark.parametrize("T,D", [(1, 1), (3, 2), (5, 17), (8, 64)])
def test_layer_norm_matches_autograd(T, D):
    x, w, b, dy, ux, uw, ub = randn(T * 100 + D, (T, D), (D,), (D,), (T, D), (T, D), (D,), (D,))
    x, w, b, dy = (t.requires_grad_() for t in (x, w, b, dy))
    eps = 1e-3
    y = torch.nn.functional.layer_norm(x, (D,), w, b, eps)
    first = torch.autograd.grad(y, (x, w, b), dy, create_graph=True)
    second = torch.autograd.grad(first, (x, w, dy), (ux, uw, ub))
    n = [t.detach().numpy() for t in (x, w, b, dy, ux, uw, ub)]
    close(om.layer_norm(n[0], n[1], n[2], eps), y)
    for a, e in zip(om.layer_norm_bwd(n[0], n[1], n[3], eps), first):
        close(a, e)
    for a, e in zip(om.layer_norm_bob(n[0], n[1], n[3], n[4], n[5], n[6], eps), second):
        close(a, e, 1e-8)  # D = 2: r^3 (v + eps small) amplifies the last bits


@pytest.mark.parametrize("T,D,V,skip", [(1, 3, 2, ()), (6, 5, 11, (0, 4)), (9, 16, 33, tuple(range(9)))])
def test_linear_ce_matches_autograd(T, D, V, skip):
    H, W, UH, UW, g = randn(T + V, (T, D), (V, D), (T, D), (V, D), (T,))
    target = torch.arange(T) * 7 % V
    target[list(skip)] = -100
    H, W, g = (t.requires_grad_() for t in (H, W, g))
    loss = torch.nn.functional.cross_entropy(H @ W.T, target, reduction="none")
    first = torch.autograd.grad(loss, (H, W), g, create_graph=True)
    second = torch.autograd.grad(first, (H, W, g), (UH, UW))
    n = [t.detach().numpy() for t in (H, W, UH, UW, g)]
    t = target.numpy()
    close(om.linear_ce(n[0], n[1], t)[0], loss)
    for a, e in zip(om.linear_ce_bwd(n[0], n[1], t, n[4]), first):
        close(a, e)
    for a, e in zip(om.linear_ce_bob(n[0], n[1], t, n[4], n[2], n[3]), second):
        close(a, e)


def test_second_order_products_match_differences():
    """<J^T u, v> = d/de <u, first backward(x + e v)> at e = 0."""
    rng = np.random.default_rng(3)
    T, D, V, h = 4, 6, 9, 1e-5
    x, dy, ux, vx, vdy = (rng.standard_normal((T, D)) for _ in range(5))
    w, uw, ub, vw = (rng.standard_normal(D) for _ in range(4))

    def f(e):
        dx, dw, db = om.layer_norm_bwd(x + e * vx, w + e * vw, dy + e * vdy, 1e-5)
        return (ux * dx).sum() + (uw * dw).sum() + (ub * db).sum()

    gx, gw, gdy = om.layer_norm_bob(x, w, dy, ux, uw, ub, 1e-5)
    assert (f(h) - f(-h)) / (2 * h) == pytest.approx((gx * vx).sum() + (gw * vw).sum() + (gdy * vdy).sum(), rel=1e-6)

    H, UH, vH = (rng.standard_normal((T, D)) for _ in range(3))
    W, UW, vW = (rng.standard_normal((V, D)) for _ in range(3))
    g, vg = rng.standard_normal(T), rng.standard_normal(T)
    t = np.array([0, -100, 8, 3])

    def f(e):
        dH, dW = om.linear_ce_bwd(H + e * vH, W + e * vW, t, g + e * vg)
        return (UH * dH).sum() + (UW * dW).sum()

    gH, gW, gg = om.linear_ce_bob(H, W, t, g, UH, UW)
    assert (f(h) - f(-h)) / (2 * h) == pytest.approx((gH * vH).sum() + (gW * vW).sum() + (gg * vg).sum(), rel=1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_rotation(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 5, 12))
    pos = np.array([[0, 1, 2, 3, 4], [7, 1000000, -3, 2 ** 31, 5]])
    theta = om.rotary_theta(8)
    y = om.rotary(x, pos, theta, interleaved)
    close((y * y).sum(-1), (x * x).sum(-1))
    close(y[..., 8:], x[..., 8:])
    close(y[0, :, 0], x[0, :, 0])                        # position 0 turns nothing
    close(om.rotary(y, pos, theta, interleaved, transpose=True), x, 1e-9)
    # the product of two rotated rows depends on their distance alone
    q, k = rng.standard_normal((2, 8))
    dot = [(om.rotary(q[None, None, None], np.array([[a]]), theta, interleaved)
            * om.rotary(k[None, None, None], np.array([[b]]), theta, interleaved)).sum() for a, b in ((3, 1), (12, 10))]
    assert dot[0] == pytest.approx(dot[1], rel=1e-9)


def test_rotary_frequencies_by_kind():
    import exact_second_order_attn_gb300 as fb
    from exact_second_order_attn_gb300.build import build
    build()
    for kind in ("none", "linear", "base", "parts"):
        for rot in (4, 64, 128):
            kw = dict(base=10000.0, scaling=kind, factor=8.0, original=8192.0, slow=1.0, fast=4.0)
            got = fb.fbob_rotary_frequencies(fb.Rotary(rot, **kw))
            ref = om.rotary_theta(rot, **kw)
            assert got == pytest.approx(ref, rel=1e-14)
    # parts: fast pairs keep their frequency, slow ones are divided by the factor
    t0 = om.rotary_theta(128)
    t = om.rotary_theta(128, scaling="parts", factor=8.0, original=8192.0)
    assert t[0] == t0[0] and t[-1] == pytest.approx(t0[-1] / 8, rel=1e-15)
    assert 8192 * t0[0] / (2 * math.pi) > 4 and 8192 * t0[-1] / (2 * math.pi) < 4
