"""Layer norm on the GPU: forward, backward and the backward's
vector-Jacobian product against the fp64 oracle."""

import numpy as np
import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from model_helpers import TYPES, check, draw, misaligned, np64

pytestmark = pytest.mark.gpu

EPS = 1e-5


def make(T, D, dtype, wtype, seed=0):
    x = draw(seed + 1, (T, D), "fp32") * (draw(seed + 2, (T, 1), "fp32").abs() + 0.5) + draw(seed + 3, (T, 1), "fp32")
    return dict(x=x.to(TYPES[dtype]), w=draw(seed + 4, (D,), wtype, 0.3, 1.0), b=draw(seed + 5, (D,), wtype, 0.3),
                dy=draw(seed + 6, (T, D), dtype), ux=draw(seed + 7, (T, D), dtype), uw=draw(seed + 8, (D,), wtype),
                ub=draw(seed + 9, (D,), wtype))


def chain(t):
    y, mean, rstd = fb.fbob_layer_norm_fwd(t["x"], t["w"], t["b"], EPS)
    dx, dw, db = fb.fbob_layer_norm_bwd(t["x"], t["w"], mean, rstd, t["dy"])
    gx, gw, gdy = fb.fbob_layer_norm_bob(t["x"], t["w"], mean, rstd, t["dy"], t["ux"], t["uw"], t["ub"])
    return dict(y=y, dx=dx, dw=dw, db=db, gx=gx, gw=gw, gdy=gdy)


def compare(t, got):
    """Roundings: a thread adds up at most 32 elements of a row, five shuffles
    and at most 32 warps follow, so a row mean carries at most 69 roundings of
    the mean magnitude, and each of the two-pass variance, the projections and
    their products uses a handful of such means: 300 of the row's largest
    magnitudes bound them all.  Column sums add the row count per thread (at
    most ceil(T / 608)), 8 warps, 19 partial rows and a shuffle tree."""
    T, D = t["x"].shape
    n = {k: np64(v) for k, v in t.items()}
    x, w, b, dy, ux, uw, ub = (n[k] for k in ("x", "w", "b", "dy", "ux", "uw", "ub"))
    mean = x.mean(-1, keepdims=True)
    r = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + EPS)
    big = lambda v: np.abs(v).max(-1, keepdims=True)  # noqa: E731
    # x's own level enters xh through x - mean, with roundings of |x| r
    xh = big(x - mean) * r + 1
    lev = big(x) * r + xh
    wm = np.abs(w).max()
    # means over a row of products with xh, bounded by rms values
    a, u, um = big(dy) * wm, big(ux), np.abs(uw).max()
    K = 300
    check("y", got["y"], om.layer_norm(x, w, b, EPS), lev * np.abs(w) + np.abs(b), K)
    dx, dw, db = om.layer_norm_bwd(x, w, dy, EPS)
    check("dx", got["dx"], dx, r * a * (1 + xh * lev), K)
    col = K + T / 8
    check("dw", got["dw"], dw, (np.abs(dy) * lev).sum(0), col)
    check("db", got["db"], db, np.abs(dy).sum(0), col)
    gx, gw, gdy = om.layer_norm_bob(x, w, dy, ux, uw, ub, EPS)
    pu = r * u * (1 + xh * lev)
    check("gdy", got["gdy"], gdy, pu * wm + um * lev + np.abs(ub), K)
    check("gw", got["gw"], gw, (pu * np.abs(dy)).sum(0), col)
    h = um * big(dy) + 2 * r * a * u * lev
    check("gx", got["gx"], gx, r * h * (1 + xh * lev) + r * r * lev * a * u * (1 + xh * lev), 2 * K)


@pytest.mark.parametrize("D", [1, 2, 3, 8, 31, 64, 255, 256, 257, 512, 520, 768, 769, 1000, 1024, 1025, 1537, 2048,
                               4096, 4100, 16384])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_layer_norm_widths(D, types):
    t = make(11, D, *types, seed=D)
    compare(t, chain(t))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 607, 609, 5000])
@pytest.mark.parametrize("D", [64, 1032])
def test_layer_norm_row_counts(T, D):
    t = make(T, D, "bf16", "fp32", seed=T)
    got = chain(t)
    compare(t, got)
    again = chain(t)
    for k in got:  # no atomics: the same bits every time
        assert torch.equal(got[k], again[k])


def test_layer_norm_misaligned_equals_aligned():
    t = make(13, 768, "bf16", "bf16")
    ref, got = chain(t), chain({k: misaligned(v) for k, v in t.items()})
    compare(t, got)
    for k in ("db",):  # the same sums in the same order
        assert torch.equal(ref[k], got[k])


@pytest.mark.parametrize("D,shift", [(769, 0), (769, 3), (1537, 1), (770, 2), (4099, 5), (8200, 1), (33, 7)])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("fp32", "fp32")])
def test_layer_norm_rows_off_bounds_touch_nothing_else(D, shift, types):
    """Rows off 16-byte bounds, all tensors shifted alike or each differently:
    the values are right, and what surrounds the outputs stays."""
    T = 37
    t = make(T, D, *types, seed=D)
    x = t["x"]

    def place(v, s, fill=5.0):
        flat = torch.full((v.numel() + 64,), fill, dtype=v.dtype, device="cuda")
        out = flat[s:s + v.numel()].view(v.shape)
        out.copy_(v)
        return flat, out

    for each in (False, True):
        s = (lambda k: (shift + k) % 8) if each else (lambda k: shift)
        u = {k: place(v, s(i))[1] for i, (k, v) in enumerate(t.items())}
        outs = {k: place(torch.zeros_like(x), s(i)) for i, k in enumerate(("y", "dx", "gx", "gdy"))}
        y, mean, rstd = fb.fbob_layer_norm_fwd(u["x"], u["w"], u["b"], EPS, y=outs["y"][1])
        dx, dw, db = fb.fbob_layer_norm_bwd(u["x"], u["w"], mean, rstd, u["dy"], dx=outs["dx"][1])
        gx, gw, gdy = fb.fbob_layer_norm_bob(u["x"], u["w"], mean, rstd, u["dy"], u["ux"], u["uw"], u["ub"],
                                             gx=outs["gx"][1], gdy=outs["gdy"][1])
        fb.device_status()
        compare(t, dict(y=y, dx=dx, dw=dw, db=db, gx=gx, gw=gw, gdy=gdy))
        for i, (k, (flat, view)) in enumerate(outs.items()):
            assert (flat[:s(i)] == 5.0).all() and (flat[s(i) + view.numel():] == 5.0).all(), k


def test_layer_norm_constant_rows_and_optional_arguments():
    """A row of equal elements has xh = 0 and r = eps^-1/2: y is the bias."""
    x = torch.full((3, 40), 2.5, device="cuda")
    b = draw(1, (40,))
    y, mean, rstd = fb.fbob_layer_norm_fwd(x, None, b, EPS)
    assert torch.equal(y, b.expand(3, 40)) and (mean == 2.5).all()
    assert rstd.cpu().numpy() == pytest.approx(EPS ** -0.5, rel=1e-6)
    t = make(6, 40, "fp32", "fp32")
    y, mean, rstd = fb.fbob_layer_norm_fwd(t["x"])
    ones, zeros = torch.ones(40, device="cuda"), torch.zeros(40, device="cuda")
    assert torch.equal(y, fb.fbob_layer_norm_fwd(t["x"], ones, zeros)[0])
    dx, dw, db = fb.fbob_layer_norm_bwd(t["x"], None, mean, rstd, t["dy"])
    full = fb.fbob_layer_norm_bwd(t["x"], ones, mean, rstd, t["dy"])
    assert dw is None and torch.equal(dx, full[0]) and torch.equal(db, full[2])
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        part = fb.fbob_layer_norm_bwd(t["x"], ones, mean, rstd, t["dy"], want=want)
        for p, f, on in zip(part, full, want):
            assert (p is None) if not on else torch.equal(p, f)
    whole = fb.fbob_layer_norm_bob(t["x"], ones, mean, rstd, t["dy"], t["ux"], zeros, zeros)
    bare = fb.fbob_layer_norm_bob(t["x"], ones, mean, rstd, t["dy"], t["ux"])
    for p, f in zip(bare, whole):
        assert torch.equal(p, f)
    part = fb.fbob_layer_norm_bob(t["x"], ones, mean, rstd, t["dy"], t["ux"], want=(False, True, False))
    assert part[0] is None and part[2] is None and torch.equal(part[1], whole[1])


def test_layer_norm_bad_rows_stay_alone():
    """NaN and infinity make their own row NaN and leave the other rows' bits."""
    t = make(20, 300, "bf16", "fp32")
    ref = chain(t)
    t["x"][4, 7], t["x"][9, 0] = float("nan"), float("inf")
    got = chain(t)
    keep = [i for i in range(20) if i not in (4, 9)]
    for k in ("y", "dx", "gx", "gdy"):
        assert torch.equal(got[k][keep], ref[k][keep]) and torch.isnan(got[k][[4, 9]]).all()


def test_layer_norm_no_rows():
    x = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(16, device="cuda")
    y, mean, rstd = fb.fbob_layer_norm_fwd(x, w, w)
    dx, dw, db = fb.fbob_layer_norm_bwd(x, w, mean, rstd, x, dw=torch.ones_like(w), db=torch.ones_like(w))
    assert y.shape == dx.shape == (0, 16) and (dw == 0).all() and (db == 0).all()
    assert (fb.fbob_layer_norm_bob(x, w, mean, rstd, x, x, gw=torch.ones_like(w))[1] == 0).all()


def test_layer_norm_streams_and_graph():
    t = make(300, 768, "bf16", "bf16")
    ref = chain(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = chain(t)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = chain(t)
    for v in held.values():
        v.fill_(9)
    g.replay()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(got[k], ref[k]) and torch.equal(held[k], ref[k])


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_layer_norm_autograd(types):
    """layer_norm's first and second derivatives are the calls' results."""
    t = make(24, 200, *types)
    ref = chain(t)
    x, w, b = (t[k].view(s).requires_grad_() for k, s in (("x", (2, 12, 200)), ("w", (200,)), ("b", (200,))))
    dy = t["dy"].view(2, 12, 200).requires_grad_()
    y = fb.layer_norm(x, w, b, EPS)
    assert torch.equal(y.view(24, 200), ref["y"])
    first = torch.autograd.grad(y, (x, w, b), dy, create_graph=True)
    for a, k in zip(first, ("dx", "dw", "db")):
        assert a.dtype == t["x" if k == "dx" else "w"].dtype and torch.equal(a.view(ref[k].shape), ref[k])
    second = torch.autograd.grad(first, (x, w, dy), (t["ux"].view(x.shape), t["uw"], t["ub"]))
    for a, k in zip(second, ("gx", "gw", "gdy")):
        assert torch.equal(a.view(ref[k].shape), ref[k])
    # only some inputs ask for a gradient, and no weight
    (only,) = torch.autograd.grad(fb.layer_norm(x.detach(), w.detach(), b, EPS), b, dy.detach())
    assert torch.equal(only, ref["db"])
    fb.layer_norm(x).sum().backward()
    assert x.grad.shape == x.shape


def test_layer_norm_against_differences():
    """The second-order product along v is the difference of first gradients."""
    t = make(5, 48, "fp32", "fp32")
    v = draw(30, (5, 48))
    h = 2.0 ** -7

    def first(e):
        x = t["x"] + e * v
        y, mean, rstd = fb.fbob_layer_norm_fwd(x, t["w"], t["b"], EPS)
        dx, dw, db = fb.fbob_layer_norm_bwd(x, t["w"], mean, rstd, t["dy"])
        return (np64(dx) * np64(t["ux"])).sum() + (np64(dw) * np64(t["uw"])).sum()

    _, mean, rstd = fb.fbob_layer_norm_fwd(t["x"], t["w"], t["b"], EPS)
    gx = fb.fbob_layer_norm_bob(t["x"], t["w"], mean, rstd, t["dy"], t["ux"], t["uw"])[0]
    exact = (np64(gx) * np64(v)).sum()
    # central differences: truncation O(h^2) of a smooth function of spread 1, rounding 2^-24 / h
    size = (np.abs(np64(gx)) * np.abs(np64(v))).sum()
    assert abs((first(h) - first(-h)) / (2 * h) - exact) <= 2e-3 * size
