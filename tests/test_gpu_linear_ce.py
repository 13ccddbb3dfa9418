"""The linear head's cross entropy on the GPU: losses, gradients and their
vector-Jacobian product against the fp64 oracle."""

import numpy as np
import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from model_helpers import U32, check, draw, half_step, misaligned, np64

pytestmark = pytest.mark.gpu


def make(T, D, V, dtype, seed=0, spread=1.5, ignored=()):
    t = dict(H=draw(seed + 1, (T, D), dtype), W=draw(seed + 2, (V, D), dtype, spread / D ** 0.5),
             UH=draw(seed + 3, (T, D), dtype), UW=draw(seed + 4, (V, D), dtype, spread / D ** 0.5),
             g=draw(seed + 5, (T,)))
    y = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed + 6))
    y[list(ignored)] = -100
    t["target"] = y.cuda()
    return t


def chain(t, **kw):
    loss, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    dH, dW = fb.fbob_linear_ce_bwd(t["H"], t["W"], t["target"], lse, t["g"], **kw)
    gH, gW, gg = fb.fbob_linear_ce_bob(t["H"], t["W"], t["target"], lse, t["g"], t["UH"], t["UW"], **kw)
    fb.device_status()
    return dict(loss=loss, lse=lse, dH=dH, dW=dW, gH=gH, gW=gW, gg=gg)


def compare(t, got):
    """Bounds, in magnitudes summed as the kernels sum them.

    A logit adds D products in fp32 (the tensor cores may drop the last bit of
    each of the D/16 steps): D/8 + 8 roundings of sum |h w| bound it; fp32
    inputs also lose the products below 2^-24 of three-term operands, within the
    same count.  An error dz of the logits moves a probability by p (2 dz + a few
    roundings of the exponent's argument, at most |z| + |lse|).  For bf16 inputs
    G and Z are rounded to bf16 once (half a step of each entry, plus the same
    again for the fp32 division by gmax, far below), up to 16 tokens to two bf16 terms."""
    n = {k: np64(v) if k != "target" else v.cpu().numpy() for k, v in t.items()}
    H, W, UH, UW, g, y = (n[k] for k in ("H", "W", "UH", "UW", "g", "target"))
    T, D = H.shape
    V = W.shape[0]
    keep = (y != -100)
    aH, aW, aUH, aUW = (np.abs(a) for a in (H * keep[:, None], W, UH * keep[:, None], UW))
    steps = D / 8 + 8
    z = (H * keep[:, None]) @ W.T
    dz = (steps * U32) * (aH @ aW.T)
    loss, lse = om.linear_ce(H, W, y)
    top = np.abs(z).max(-1) + np.abs(lse)
    wander = dz.max(-1) + 16 * U32 * (top + np.log(V) + 1)
    check("loss", got["loss"], loss, 0, 0, extra=keep * 2 * wander)
    check("lse", got["lse"], lse, 0, 0, extra=keep * 2 * wander)
    q = U32
    if t["H"].dtype == torch.bfloat16:  # one bf16 term, two up to 16 tokens
        q = half_step(torch.bfloat16) if T > 16 else half_step(torch.bfloat16) ** 2
    p = np.exp(z - lse[:, None]) * keep[:, None]
    one = np.zeros_like(p)
    one[np.nonzero(keep)[0], y[keep]] = 1
    ag = np.abs(g)[:, None]
    G = ag * np.abs(p - one)
    dp = p * (4 * wander[:, None])
    dG = ag * dp + 1.01 * q * G + 4 * U32 * ag * (p + one)
    dH, dW = om.linear_ce_bwd(H, W, y, g)
    sv, st = V / 8 + 64, T / 8 + 64   # roundings of the sums over classes and tokens
    check("dH", got["dH"], dH, G @ aW, sv, extra=dG @ aW)
    check("dW", got["dW"], dW, G.T @ aH, st, extra=dG.T @ aH)
    b = np.abs((UH * keep[:, None]) @ W.T + (H * keep[:, None]) @ UW.T)
    db = 2 * steps * U32 * (aUH @ aW.T + aH @ aUW.T)
    alpha = (p * b).sum(-1, keepdims=True)  # of magnitudes
    dalpha = (dp * b + p * db).sum(-1, keepdims=True) + (V / 64 + 64) * U32 * alpha
    gH, gW, gg = om.linear_ce_bob(H, W, y, g, UH, UW)
    check("gg", got["gg"], gg, (alpha + (one * b).sum(-1, keepdims=True))[:, 0], 4,
          extra=(dalpha + db.max(-1, keepdims=True))[:, 0])
    true_alpha = (p * ((UH * keep[:, None]) @ W.T + (H * keep[:, None]) @ UW.T)).sum(-1, keepdims=True)
    centred = np.abs((UH * keep[:, None]) @ W.T + (H * keep[:, None]) @ UW.T - true_alpha)
    Z = ag * p * centred
    dZ = ag * (dp * centred + p * (db + dalpha + 4 * U32 * (b + np.abs(true_alpha)))) + 1.01 * q * Z
    check("gH", got["gH"], gH, Z @ aW + G @ aUW, 2 * sv, extra=dZ @ aW + dG @ aUW)
    check("gW", got["gW"], gW, Z.T @ aH + G.T @ aUH, 2 * st, extra=dZ.T @ aH + dG.T @ aUH)


@pytest.mark.parametrize("T,D,V", [(1, 8, 1), (1, 16, 2), (3, 64, 127), (128, 64, 128), (129, 72, 129), (255, 128, 255),
                                   (256, 256, 256), (257, 320, 257), (300, 768, 1000), (24, 768, 5003), (2, 1032, 513),
                                   (700, 40, 600), (5, 16, 40007)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_ce_against_oracle(T, D, V, dtype):
    t = make(T, D, V, dtype, seed=T + V, ignored=range(0, T, 5) if T > 1 else ())
    compare(t, chain(t))


@pytest.mark.parametrize("D", [1, 3, 4, 7, 12, 36, 65, 130, 396])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_ce_odd_widths(D, dtype):
    """Widths that the padding rounds up: right values, nothing written past
    the outputs."""
    t = make(37, D, 301, dtype, seed=D)
    compare(t, chain(t))
    _, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    flat = [torch.full((x.numel() + 64,), 9.0, dtype=x.dtype, device="cuda") for x in (t["H"], t["W"])]
    dH, dW = (f[:x.numel()].view(x.shape) for f, x in zip(flat, (t["H"], t["W"])))
    fb.fbob_linear_ce_bwd(t["H"], t["W"], t["target"], lse, t["g"], dH=dH, dW=dW)
    fb.fbob_linear_ce_bob(t["H"], t["W"], t["target"], lse, t["g"], t["UH"], t["UW"], gH=dH, gW=dW)
    for f in flat:
        assert (f[-64:] == 9.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_ce_pieces(dtype):
    """Any cut of the vocabulary gives the gradients; dW, which no cut sums
    over, has the same bits."""
    t = make(200, 64, 1500, dtype, seed=9, ignored=(1, 2, 199))
    whole = chain(t)
    for piece in (1, 256, 700, 1500):
        got = chain(t, piece=piece)
        compare(t, got)
        assert torch.equal(got["dW"], whole["dW"]) and torch.equal(got["gW"], whole["gW"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,piece", [(5121, 1280), (5 * 1280, 1280), (20481, 5120), (2049, 2048)])
def test_linear_ce_short_last_piece(dtype, V, piece):
    """A last piece of one class, after pieces whose contraction is cut into
    several slabs."""
    t = make(9, 32, V, dtype, seed=V)
    compare(t, chain(t, piece=piece))


def test_linear_ce_peaked_rows():
    """Targets that hold nearly all of the probability, and others none."""
    t = make(150, 128, 700, "bf16", seed=21, spread=12.0)
    top = (t["H"].float() @ t["W"].float().T).argmax(-1)
    t["target"][::2] = top[::2]
    compare(t, chain(t))


def test_linear_ce_ignored_tokens_hold_anything():
    """NaN and infinities in ignored tokens (and their g, UH) reach nothing."""
    bad = (0, 5, 6, 40)
    t = make(41, 96, 333, "bf16", seed=4, ignored=bad)
    ref = chain(t)
    compare(t, ref)
    for i, v in zip(bad, (float("nan"), float("inf"), -float("inf"), float("nan"))):
        t["H"][i], t["UH"][i], t["g"][i] = v, v, v
    got = chain(t)
    for k in ref:
        assert torch.equal(got[k], ref[k]), k
    for k in ("loss", "lse", "dH", "gH", "gg"):
        assert (got[k][list(bad)] == 0).all()


def test_linear_ce_all_ignored_and_no_tokens():
    t = make(9, 64, 50, "bf16", ignored=range(9))
    for k, v in chain(t).items():
        assert (v == 0).all(), k
    H = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, z = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = fb.fbob_linear_ce_fwd(H, t["W"], y)
    dH, dW = fb.fbob_linear_ce_bwd(H, t["W"], y, lse, z, dW=torch.ones_like(t["W"]))
    assert loss.shape == (0,) and dH.shape == (0, 64) and (dW == 0).all()
    gH, gW, gg = fb.fbob_linear_ce_bob(H, t["W"], y, lse, z, H, t["UW"], gW=torch.ones_like(t["W"]))
    assert gH.shape == (0, 64) and (gW == 0).all() and gg.shape == (0,)


@pytest.mark.parametrize("T,counted", [(9000, 8999), (9000, 1), (40000, 39000), (5000, 64), (4097, 65), (300, 256), (300, 257)])
def test_linear_ce_counts_of_tokens(T, counted):
    """Lists of counted tokens over several rounds, and at the steps' edges."""
    order = torch.randperm(T, generator=torch.Generator().manual_seed(T))
    t = make(T, 16, 40, "bf16", seed=counted, ignored=order[counted:].tolist())
    compare(t, chain(t))


@pytest.mark.parametrize("wrong", [-1, 50, 2 ** 40])
def test_linear_ce_target_outside_the_classes(wrong):
    t = make(9, 64, 50, "bf16", seed=2)
    t["target"][4] = -100
    ref = chain(t)
    t["target"][4] = wrong
    loss, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    with pytest.raises(fb.FbobError, match="INVALID_ARG"):
        fb.device_status()
    assert torch.isnan(loss[4]) and torch.equal(loss[:4], ref["loss"][:4])
    dH, dW = fb.fbob_linear_ce_bwd(t["H"], t["W"], t["target"], lse, t["g"])
    with pytest.raises(fb.FbobError, match="INVALID_ARG"):
        fb.device_status()
    assert torch.equal(dH, ref["dH"]) and torch.equal(dW, ref["dW"])
    t["target"][4] = -100
    fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    fb.device_status()  # cleared


def test_linear_ce_nan_logits_stay_in_their_token():
    t = make(20, 64, 300, "bf16", seed=8)
    ref = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    t["H"][3, 5] = float("nan")
    t["H"][11, 0] = float("inf")
    loss, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    keep = [i for i in range(20) if i not in (3, 11)]
    assert torch.equal(loss[keep], ref[0][keep]) and torch.isnan(loss[[3, 11]]).all()
    fb.device_status()


@pytest.mark.parametrize("g", ["equal", "zero", "tiny", "huge", "one"])
def test_linear_ce_scales_of_g(g):
    t = make(60, 64, 400, "bf16", seed=13)
    t["g"] = {"equal": torch.full((60,), 1 / 61.0), "zero": torch.zeros(60), "tiny": torch.full((60,), 1e-30),
              "huge": torch.full((60,), 1e25), "one": torch.nn.functional.one_hot(torch.tensor(7), 60).float()}[g].cuda()
    compare(t, chain(t))


def test_linear_ce_wanted_outputs_and_missing_cotangents():
    t = make(70, 64, 500, "bf16", seed=3)
    full = chain(t)
    lse, a = full["lse"], (t["H"], t["W"], t["target"])
    for want in ((True, False), (False, True), (False, False)):
        part = fb.fbob_linear_ce_bwd(*a, lse, t["g"], want=want)
        for p, k, on in zip(part, ("dH", "dW"), want):
            assert (p is None) if not on else torch.equal(p, full[k])
    for want in ((True, False, False), (False, True, False), (False, False, True)):
        part = fb.fbob_linear_ce_bob(*a, lse, t["g"], t["UH"], t["UW"], want=want)
        for p, k, on in zip(part, ("gH", "gW", "gg"), want):
            assert (p is None) if not on else torch.equal(p, full[k])
    for gone in ("UH", "UW"):
        u = dict(UH=t["UH"], UW=t["UW"])
        zero = {**u, gone: torch.zeros_like(u[gone])}
        u[gone] = None
        for p, f in zip(fb.fbob_linear_ce_bob(*a, lse, t["g"], u["UH"], u["UW"]),
                        fb.fbob_linear_ce_bob(*a, lse, t["g"], zero["UH"], zero["UW"])):
            assert torch.equal(p, f)
    with pytest.raises(fb.FbobError):
        fb.fbob_linear_ce_bob(*a, lse, t["g"], None, None)


def test_linear_ce_alignment_repeats_and_graph():
    t = make(130, 64, 900, "fp32", seed=6)
    ref = chain(t)
    odd = {k: misaligned(v) if k not in ("target",) else v for k, v in t.items()}
    got = chain(odd)
    again = chain(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = chain(t)
    for k in ref:
        assert torch.equal(ref[k], got[k]) and torch.equal(ref[k], again[k]) and torch.equal(ref[k], side[k]), k
    t16 = {k: v.bfloat16() if k in ("H", "W", "UH", "UW") else v for k, v in t.items()}
    out = torch.empty(130 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(130, 64)
    _, lse = fb.fbob_linear_ce_fwd(misaligned(t16["H"]), t16["W"], t16["target"])
    a = fb.fbob_linear_ce_bwd(misaligned(t16["H"]), t16["W"], t16["target"], lse, t16["g"], dH=out)
    b = fb.fbob_linear_ce_bwd(t16["H"], t16["W"], t16["target"], lse, t16["g"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(fb.FbobError, match="aligned"):
        fb.fbob_linear_ce_fwd(t16["H"], misaligned(t16["W"]), t16["target"])
    # captured: a replay works on the values of its own time
    g = torch.cuda.CUDAGraph()
    loss, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
    with torch.cuda.graph(g):
        loss, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
        dH, dW = fb.fbob_linear_ce_bwd(t["H"], t["W"], t["target"], lse, t["g"])
        gH, gW, gg = fb.fbob_linear_ce_bob(t["H"], t["W"], t["target"], lse, t["g"], t["UH"], t["UW"])
    t["H"].mul_(-1)
    t["target"][3] = -100
    g.replay()
    torch.cuda.synchronize()
    held = dict(loss=loss, lse=lse, dH=dH, dW=dW, gH=gH, gW=gW, gg=gg)
    for k, v in chain(t).items():
        assert torch.equal(v, held[k]), k


def test_linear_ce_given_workspace_and_refusals():
    t = make(33, 64, 300, "bf16", seed=1)
    full = chain(t)
    for which, call in ((0, lambda w: fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"], workspace=w)[0]),
                        (1, lambda w: fb.fbob_linear_ce_bwd(t["H"], t["W"], t["target"], full["lse"], t["g"], workspace=w)[1]),
                        (2, lambda w: fb.fbob_linear_ce_bob(t["H"], t["W"], t["target"], full["lse"], t["g"], t["UH"], t["UW"], workspace=w)[1])):
        need = fb.fbob_linear_ce_workspace_bytes(fb.linear_ce_for(t["H"], t["W"]), which)
        guard = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(guard[:need]), full[("loss", "dW", "gW")[which]])
        assert (guard[need:] == 255).all()
        with pytest.raises(fb.FbobError, match="WORKSPACE"):
            call(guard[:need - 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_ce_autograd(dtype):
    t = make(50, 64, 300, dtype, seed=17, ignored=(7,))
    ref = chain(t)
    H, W, g = (t[k].requires_grad_() for k in ("H", "W", "g"))
    loss = fb.linear_cross_entropy(H, W, t["target"])
    assert torch.equal(loss, ref["loss"])
    dH, dW = torch.autograd.grad(loss, (H, W), g, create_graph=True)
    assert torch.equal(dH, ref["dH"]) and torch.equal(dW, ref["dW"])
    for a, k in zip(torch.autograd.grad((dH, dW), (H, W, g), (t["UH"], t["UW"])), ("gH", "gW", "gg")):
        assert torch.equal(a, ref[k])
    # a mean loss hands over an expanded gradient
    (dm,) = torch.autograd.grad(fb.linear_cross_entropy(H, W.detach(), t["target"]).mean(), H)
    assert dm.shape == H.shape and (dm[7] == 0).all()


def test_linear_ce_against_differences():
    """First gradients against differences of the loss, second ones against
    differences of first gradients, along a direction (fp32)."""
    t = make(12, 32, 90, "fp32", seed=31)
    vH, vW = draw(40, (12, 32)), draw(41, (90, 32), std=0.2)
    h = 2.0 ** -6

    def at(e):
        H, W = t["H"] + e * vH, t["W"] + e * vW
        loss, lse = fb.fbob_linear_ce_fwd(H, W, t["target"])
        dH, dW = fb.fbob_linear_ce_bwd(H, W, t["target"], lse, t["g"])
        return (np64(loss) * np64(t["g"])).sum(), (np64(dH) * np64(t["UH"])).sum() + (np64(dW) * np64(t["UW"])).sum()

    r = chain(t)
    (l1, f1), (l0, f0) = at(h), at(-h)
    first = (np64(r["dH"]) * np64(vH)).sum() + (np64(r["dW"]) * np64(vW)).sum()
    second = (np64(r["gH"]) * np64(vH)).sum() + (np64(r["gW"]) * np64(vW)).sum()
    size1 = np.abs(np64(r["dH"]) * np64(vH)).sum() + np.abs(np64(r["dW"]) * np64(vW)).sum()
    size2 = np.abs(np64(r["gH"]) * np64(vH)).sum() + np.abs(np64(r["gW"]) * np64(vW)).sum()
    # h^2 / 6 of third derivatives of order one, and fp32 roundings over h
    assert abs((l1 - l0) / (2 * h) - first) <= 1e-3 * size1
    assert abs((f1 - f0) / (2 * h) - second) <= 2e-3 * size2


def test_linear_ce_timeout_is_reported():
    """A producer that withholds its first stage: the kernels give up, return
    and set the status; the next call works."""
    t = make(300, 128, 600, "bf16", seed=5)
    ref = chain(t)
    old = fb.fbob_set_wait_limit_ns(2_000_000)
    fb.fbob_debug_stall_producer(True)
    try:
        fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
        with pytest.raises(fb.FbobError, match="TIMEOUT"):
            fb.device_status()
    finally:
        fb.fbob_debug_stall_producer(False)
        fb.fbob_set_wait_limit_ns(old)
    got = chain(t)
    for k in ref:
        assert torch.equal(got[k], ref[k])
