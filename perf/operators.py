"""The operators of a model around the attention, as cases that can be timed and compared.

Three operators, each differentiable twice like the attention they surround:

* rotary positions on Q and K (forward, and its transpose for the gradients);
* layer norm (forward, backward with the weight's and bias's gradients, and the backward's own
  vector-Jacobian product);
* the softmax cross entropy of a linear head (per-token losses without stored logits, the
  gradients of the hidden states and the head, and their own vector-Jacobian product).

``run`` computes a case either in plain torch operations in 32 bits (``own = False``) or through
this package's entry points (``own = True``); ``exact`` gives the same values in 64 bits.

Formulas (one row of layer norm has D elements; m() is the mean over a row):

  rotary       y = m_s [cos -sin; sin cos] x per pair, angle = position * theta_i;
               theta_i = base^(-2i/rot), scaled by kind:
               linear  theta / factor
               base    base * factor^(rot/(rot-2)) in place of base
               parts   theta * (w + (1-w)/factor), w = clamp((n - slow)/(fast - slow), 0, 1),
                       n = original * theta / 2 pi, the turns within the original length
  layer norm   y = w xh + b, xh = (x - m(x)) r, r = (m((x - m(x))^2) + eps)^(-1/2)
  head loss    z = W h, loss = log sum_v exp z_v - z_target (0 where the target is ignored)
"""

from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGNORE = -100


def listed():
    return [
        # A token appended to each of eight sequences: one position, latency only.
        dict(name="rotary_one_token", op="rotary", step="fwd", B=8, H=12, Hk=12, N=1, d=64, rot=64, interleaved=False,
             scaling="none", offset=1023, packed=True, dtype="bf16"),
        # GPT-2-Small-shaped training step: Q and K read out of a packed projection, gradients
        # written back into one.
        dict(name="rotary_gpt2s_step", op="rotary", step="step", B=8, H=12, Hk=12, N=1024, d=64, rot=64,
             interleaved=False, scaling="none", offset=0, packed=True, dtype="bf16"),
        # The wide-head configuration (2 x 16 heads, 16,384 tokens), neighbouring pairs, half of
        # the head rotated, frequencies scaled by parts for a context beyond the original one.
        dict(name="rotary_wide_long", op="rotary", step="step", B=2, H=16, Hk=16, N=16384, d=128, rot=64,
             interleaved=True, scaling="parts", offset=1000000, packed=False, dtype="bf16"),
        # The norm of one new token per sequence.
        dict(name="norm_few_rows", op="norm", step="fwd", T=8, D=768, dtype="bf16", wtype="bf16"),
        # GPT-2-Small-shaped step: eight sequences of 1024 tokens, forward and backward.
        dict(name="norm_gpt2s_step", op="norm", step="step", T=8192, D=768, dtype="bf16", wtype="bf16"),
        # The same inside a Hessian-vector product; weights kept in 32 bits.
        dict(name="norm_gpt2s_second", op="norm", step="second", T=8192, D=768, dtype="bf16", wtype="fp32"),
        # 32 heads of 128 columns, 4 sequences of 8192 tokens (the peaky configuration's model).
        dict(name="norm_wide_step", op="norm", step="step", T=32768, D=4096, dtype="bf16", wtype="bf16"),
        # Odd sizes in 32 bits, through the second order.
        dict(name="norm_odd_fp32", op="norm", step="second", T=5003, D=1537, dtype="fp32", wtype="fp32"),
        # The loss of a handful of scored tokens: reading the head bounds it.
        dict(name="loss_few_tokens", op="loss", step="step", T=24, D=768, V=50257, ignored=0.0, dtype="bf16"),
        # GPT-2-Small-shaped training step, a tenth of the tokens ignored (prompts, padding).
        dict(name="loss_gpt2s_step", op="loss", step="step", T=8192, D=768, V=50257, ignored=0.1, dtype="bf16"),
        # Its Hessian-vector product on half the tokens.
        dict(name="loss_gpt2s_second", op="loss", step="second", T=4096, D=768, V=50257, ignored=0.1, dtype="bf16"),
        # A small model in 32 bits, odd vocabulary and token count.
        dict(name="loss_fp32_step", op="loss", step="step", T=1021, D=512, V=32003, ignored=0.05, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "loss"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "rotary":
        d = rng.choice([32, 64, 96, 128])
        H = rng.randint(1, 32)
        Hk = rng.choice([H, max(1, H // 4)])
        B = rng.randint(1, 8)
        N = _log(rng, 1, max(1, min(65536, (2 ** 26) // (B * H * d))))
        rot = rng.choice([d, d, d // 2])
        return dict(op=op, step=rng.choice(["fwd", "step"]), B=B, H=H, Hk=Hk, N=N, d=d, rot=rot,
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "parts"]),
                    offset=rng.choice([0, rng.randint(0, 2 ** 20)]), packed=rng.random() < 0.5, dtype=dtype)
    if op == "norm":
        D = rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 8, 1024)])
        T = _log(rng, 1, max(1, min(65536, (2 ** 26) // D)))
        return dict(op=op, step=rng.choice(["fwd", "step", "second"]), T=T, D=D, dtype=dtype,
                    wtype=rng.choice(["fp32", dtype]))
    D = 8 * _log(rng, 8, 256)
    V = _log(rng, 257, 65536)
    T = _log(rng, 1, max(1, min(8192, (2 ** 37 if dtype == "bf16" else 2 ** 34) // (V * D))))
    return dict(op=op, step=rng.choice(["fwd", "step", "second"]), T=T, D=D, V=V,
                ignored=rng.choice([0.0, 0.1, 0.5]), dtype=dtype)


# --- what a user's program holds -------------------------------------------------------------

_BASE = 10000.0


def _scaling(case):
    """(factor, original length, slow, fast, magnitude) of a case's rotary scaling."""
    if case["scaling"] == "none":
        return 1.0, 0.0, 0.0, 0.0, 1.0
    return 8.0, 8192.0, 1.0, 4.0, (1.0 if case["scaling"] != "parts" else 1.2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return x.mul_(std).add_(mean).to(dtype)

    s = dict(case)
    if case["op"] == "rotary":
        B, H, Hk, N, d = (case[k] for k in ("B", "H", "Hk", "N", "d"))
        if case["packed"]:  # Q, K and V of a token side by side, as a joint projection leaves them
            qkv = normal(B, N, H + 2 * Hk, d)
            s["Q"] = qkv[:, :, :H].transpose(1, 2)
            s["K"] = qkv[:, :, H:H + Hk].transpose(1, 2)
        else:
            s["Q"], s["K"] = normal(B, H, N, d), normal(B, Hk, N, d)
        # each sequence at its own place
        starts = torch.randint(0, 64, (B, 1), generator=g, device="cuda") + case["offset"]
        s["positions"] = starts + torch.arange(N, device="cuda")
        if case["step"] == "step":
            s["dQ"], s["dK"] = normal(B, H, N, d, std=0.1), normal(B, Hk, N, d, std=0.1)
        factor, original, slow, fast, magnitude = _scaling(case)
        if own:  # the description of the rotation (no data), which a model keeps
            import exact_second_order_attn_gb300 as fb
            s["rotary"] = fb.Rotary(case["rot"], base=_BASE, interleaved=case["interleaved"], scaling=case["scaling"],
                                    factor=factor, original=original, slow=slow, fast=fast, magnitude=magnitude)
        return s
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        wt = _TYPES[case["wtype"]]
        # a residual stream: a common level per row, rows of different spread
        spread = torch.rand(T, 1, generator=g, device="cuda") * 2 + 0.5
        s["x"] = (normal(T, D, dtype=torch.float32) * spread + normal(T, 1, std=0.3, dtype=torch.float32)).to(dt)
        s["w"], s["b"] = normal(D, std=0.2, mean=1.0, dtype=wt), normal(D, std=0.2, dtype=wt)
        if case["step"] != "fwd":
            s["dy"] = normal(T, D, std=0.1)
        if case["step"] == "second":
            s["ux"], s["uw"], s["ub"] = normal(T, D), normal(D, dtype=wt), normal(D, dtype=wt)
        return s
    T, D, V = case["T"], case["D"], case["V"]
    s["h"], s["W"] = normal(T, D), normal(V, D, std=2.0 / math.sqrt(D))
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    skip = torch.rand(T, generator=g, device="cuda") < case["ignored"]
    s["target"] = torch.where(skip, IGNORE, target)
    # the gradient of a mean over the scored tokens
    s["g"] = torch.full((T,), 1.0, device="cuda") / (~skip).sum().clamp(min=1)
    if case["step"] == "second":
        s["uh"], s["uw"] = normal(T, D), normal(V, D, std=2.0 / math.sqrt(D))
    return s


# --- plain forms --------------------------------------------------------------------------------

def _angles(case, positions):
    """cos and sin [B, 1, N, rot / 2] in 32 bits; angles in 64 (positions reach a million)."""
    rot = case["rot"]
    factor, original, slow, fast, magnitude = _scaling(case)
    base = _BASE
    if case["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, device=positions.device, dtype=torch.float64)
    theta = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        theta = theta / factor
    if case["scaling"] == "parts":
        w = ((original * theta / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        theta = theta * (w + (1 - w) / factor)
    a = positions[:, None, :, None].double() * theta
    return (a.cos() * magnitude).float(), (a.sin() * magnitude).float()


def _rotate(case, x, cos, sin):
    rot, half = case["rot"], case["rot"] // 2
    f = x.float()
    if case["interleaved"]:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:rot]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, f[..., rot:]), -1).to(x.dtype)


def _plain_rotary(s):
    cos, sin = _angles(s, s["positions"])
    out = {"q": _rotate(s, s["Q"], cos, sin), "k": _rotate(s, s["K"], cos, sin)}
    if s["step"] == "step":
        out["dq"] = _rotate(s, s["dQ"], cos, -sin)
        out["dk"] = _rotate(s, s["dK"], cos, -sin)
    return out


def _plain_norm(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5)
    xh = c * r
    out = {"y": (xh * w + b).to(s["x"].dtype)}
    if s["step"] == "fwd":
        return out
    dy = s["dy"].float()
    a = dy * w
    ma, max_ = a.mean(-1, keepdim=True), (a * xh).mean(-1, keepdim=True)
    out["dx"] = (r * (a - ma - xh * max_)).to(s["x"].dtype)
    out["dw"] = (dy * xh).sum(0).to(s["w"].dtype)
    out["db"] = dy.sum(0).to(s["w"].dtype)
    if s["step"] == "step":
        return out
    # vector-Jacobian product of (dx, dw, db) as functions of (x, w, dy)
    u, uw, ub = s["ux"].float(), s["uw"].float(), s["ub"].float()
    mu, mux = u.mean(-1, keepdim=True), (u * xh).mean(-1, keepdim=True)
    pu = u - mu - xh * mux
    out["gdy"] = (r * w * pu + uw * xh + ub).to(s["x"].dtype)
    out["gw"] = (r * pu * dy).sum(0).to(s["w"].dtype)
    h = uw * dy - r * (a * mux + u * max_)
    mh, mhx = h.mean(-1, keepdim=True), (h * xh).mean(-1, keepdim=True)
    s1 = (pu * a).mean(-1, keepdim=True)
    out["gx"] = (r * (h - mh - xh * mhx) - r * r * xh * s1).to(s["x"].dtype)
    return out


def _plain_loss(s):
    dt = s["h"].dtype
    keep = s["target"] != IGNORE
    y = torch.where(keep, s["target"], 0)[:, None]
    h, W = torch.where(keep[:, None], s["h"], 0).float(), s["W"].float()
    z = h @ W.T
    top = z.max(-1, keepdim=True).values
    lse = (z - top).exp().sum(-1, keepdim=True).log() + top
    out = {"loss": torch.where(keep, (lse - z.gather(1, y))[:, 0], 0)}
    if s["step"] == "fwd":
        return out
    g = torch.where(keep, s["g"], 0)[:, None]
    p = (z - lse).exp()
    G = p * g
    G.scatter_add_(1, y, -g)
    out["dh"], out["dW"] = (G @ W).to(dt), (G.T @ h).to(dt)
    if s["step"] == "step":
        return out
    # vector-Jacobian product of (dh, dW) as functions of (h, W, g)
    uh, uW = torch.where(keep[:, None], s["uh"], 0).float(), s["uw"].float()
    b = uh @ W.T + h @ uW.T
    alpha = (p * b).sum(-1, keepdim=True)
    out["gg"] = torch.where(keep, (alpha - b.gather(1, y))[:, 0], 0)
    Z = g * p * (b - alpha)
    out["gh"] = (Z @ W + G @ uW).to(dt)
    out["gW"] = (Z.T @ h + G.T @ uh).to(dt)
    return out


# --- the framework's calls ----------------------------------------------------------------------

def _own_rotary(fb, s):
    r, pos = s["rotary"], s["positions"]
    q, k = fb.fbob_rotary_apply(r, s["Q"], s["K"], positions=pos)
    out = {"q": q, "k": k}
    if s["step"] == "step":
        dq = dk = None
        if s["packed"]:  # gradients side by side, as the joint projection's backward reads them
            B, H, Hk, N, d = (s[n] for n in ("B", "H", "Hk", "N", "d"))
            dqk = torch.empty(B, N, H + Hk, d, dtype=s["Q"].dtype, device=s["Q"].device)
            dq, dk = dqk[:, :, :H].transpose(1, 2), dqk[:, :, H:].transpose(1, 2)
        out["dq"], out["dk"] = fb.fbob_rotary_apply(r, s["dQ"], s["dK"], positions=pos, transpose=True, Qo=dq, Ko=dk)
    return out


def _own_norm(fb, s):
    y, mean, rstd = fb.fbob_layer_norm_fwd(s["x"], s["w"], s["b"], 1e-5)
    out = {"y": y}
    if s["step"] != "fwd":
        out["dx"], out["dw"], out["db"] = fb.fbob_layer_norm_bwd(s["x"], s["w"], mean, rstd, s["dy"])
    if s["step"] == "second":
        out["gx"], out["gw"], out["gdy"] = fb.fbob_layer_norm_bob(s["x"], s["w"], mean, rstd, s["dy"], s["ux"],
                                                                  s["uw"], s["ub"])
    return out


def _own_loss(fb, s):
    loss, lse = fb.fbob_linear_ce_fwd(s["h"], s["W"], s["target"], ignore_index=IGNORE)
    out = {"loss": loss}
    if s["step"] != "fwd":
        out["dh"], out["dW"] = fb.fbob_linear_ce_bwd(s["h"], s["W"], s["target"], lse, s["g"], ignore_index=IGNORE)
    if s["step"] == "second":
        out["gh"], out["gW"], out["gg"] = fb.fbob_linear_ce_bob(s["h"], s["W"], s["target"], lse, s["g"], s["uh"],
                                                                s["uw"], ignore_index=IGNORE)
    return out


def run(state):
    op = state["op"]
    if own:
        import exact_second_order_attn_gb300 as fb
        return {"rotary": _own_rotary, "norm": _own_norm, "loss": _own_loss}[op](fb, state)
    return {"rotary": _plain_rotary, "norm": _plain_norm, "loss": _plain_loss}[op](state)


# --- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        n = case["B"] * case["N"] * case["d"] * (case["H"] + case["Hk"])
        turns = 2 if case["step"] == "step" else 1
        # in and out each way, one position per token; a rotated pair costs four products, two sums
        return dict(bytes=turns * (2 * n * e + 8 * case["B"] * case["N"]),
                    flops=turns * 3 * n * case["rot"] / case["d"])
    if case["op"] == "norm":
        n, D = case["T"] * case["D"], case["D"]
        we = 2 if case["wtype"] == "bf16" else 4
        # big tensors in and out: x, y; dy, dx; ux, gx, gdy
        big, vec, fl = {"fwd": (2, 2, 8), "step": (4, 4, 20), "second": (7, 7, 45)}[case["step"]]
        return dict(bytes=big * n * e + vec * D * we, flops=fl * n)
    T, D, V = case["T"], case["D"], case["V"]
    h, w = T * D * e, V * D * e
    # products of 2 T D V each: the logits; dh, dW; the cotangent's logits (2), gh (2), gW (2)
    products = {"fwd": 1, "step": 3, "second": 9}[case["step"]]
    bytes_ = {"fwd": h + w + 12 * T, "step": 2 * (h + w) + 16 * T, "second": 4 * (h + w) + 20 * T}[case["step"]]
    return dict(bytes=bytes_, flops=products * 2 * T * D * V)


# --- 64 bits --------------------------------------------------------------------------------------

def _exact_rotary(case, s):
    rot = case["rot"]
    factor, original, slow, fast, magnitude = _scaling(case)
    theta = []
    for i in range(rot // 2):
        base = _BASE * (factor ** (rot / (rot - 2)) if case["scaling"] == "base" else 1.0)
        t = math.exp(-math.log(base) * 2 * i / rot)
        if case["scaling"] == "linear":
            t /= factor
        elif case["scaling"] == "parts":
            n = original * t / (2 * math.pi)
            w = 0.0 if n <= slow else 1.0 if n >= fast else (n - slow) / (fast - slow)
            t = w * t + (1 - w) * t / factor
        theta.append(t)
    turn = torch.polar(torch.tensor(magnitude, dtype=torch.float64, device="cuda"),
                       s["positions"].double()[..., None] * torch.tensor(theta, dtype=torch.float64, device="cuda"))
    turn = turn[:, None]  # [B, 1, N, rot / 2]

    def spin(x, turn):
        x = x.double()
        head, tail = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            z = torch.complex(*head.reshape(*head.shape[:-1], rot // 2, 2).unbind(-1)) * turn
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(*head.reshape(*head.shape[:-1], 2, rot // 2).unbind(-2)) * turn
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, tail), -1)

    out = {"q": spin(s["Q"], turn), "k": spin(s["K"], turn)}
    if case["step"] == "step":
        out["dq"], out["dk"] = spin(s["dQ"], turn.conj()), spin(s["dK"], turn.conj())
    return out


def _exact_norm(case, s):
    x, w, b = (s[k].double().requires_grad_(case["step"] != "fwd") for k in ("x", "w", "b"))
    var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
    y = (x - mean) / (var + 1e-5).sqrt() * w + b
    out = {"y": y.detach()}
    if case["step"] == "fwd":
        return out
    second = case["step"] == "second"
    dy = s["dy"].double().requires_grad_(second)
    got = torch.autograd.grad(y, [x, w, b], dy, create_graph=second)
    out |= dict(zip(("dx", "dw", "db"), (t.detach() for t in got)))
    if second:
        u = [s[k].double() for k in ("ux", "uw", "ub")]
        out |= dict(zip(("gx", "gw", "gdy"), torch.autograd.grad(got, [x, w, dy], u)))
    return out


def _exact_loss(case, s):
    rows = (s["target"] != IGNORE).nonzero()[:, 0]
    T, D = s["h"].shape
    grad = case["step"] != "fwd"
    h, W = s["h"][rows].double().requires_grad_(grad), s["W"].double().requires_grad_(grad)
    y = s["target"][rows]

    def whole(x):
        return torch.zeros(T, *x.shape[1:], dtype=x.dtype, device=x.device).index_copy_(0, rows, x)

    loss = -torch.log_softmax(torch.matmul(h, W.t()), -1)[torch.arange(len(rows), device=y.device), y]
    out = {"loss": whole(loss.detach())}
    if not grad:
        return out
    second = case["step"] == "second"
    g = s["g"][rows].double().requires_grad_(second)
    got = torch.autograd.grad(loss, [h, W], g, create_graph=second)
    out |= {"dh": whole(got[0].detach()), "dW": got[1].detach()}
    if second:
        gh, gW, gg = torch.autograd.grad(got, [h, W, g], [s["uh"][rows].double(), s["uw"].double()])
        out |= {"gh": whole(gh), "gW": gW, "gg": whole(gg)}
    return out


def exact(case, seed):
    if case["op"] == "loss" and work(case)["flops"] > 8e12:  # over about 20 s in 64 bits
        return None
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "norm": _exact_norm, "loss": _exact_loss}[case["op"]](case, s)
