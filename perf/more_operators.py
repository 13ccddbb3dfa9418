"""Linear layers and dropout as cases that can be timed and compared.

Two operators, differentiable twice like the attention they feed:

* the matrix product of a linear layer with bias, activation, dropout and residual in its
  epilogue (forward, backward, and the backward's own vector-Jacobian product);
* dropout whose mask comes from a counter-based generator and is never stored, alone or added
  to a residual.

``run`` computes a case either in plain torch operations in 32 bits (``own = False``) or through
this package's entry points (``own = True``); ``exact`` gives the same values in 64 bits.

Formulas (x [T, K], W [N, K]; a the activation, m the dropout factor of an element):

  linear   z = x W^T + b, y = r + m a(z)
           dz = m dy a'(z), dx = dz W, dW = dz^T x, db = sum over rows of dz
           along (ux, uW, ub): t = ux W^T + x uW^T + ub, q = m t dy a''(z),
           gdy = m t a'(z), gx = q W + dz uW, gW = q^T x + dz^T ux, gb = sum over rows of q
  dropout  y = r + m x, dx = m dy
  m        element (row, column): n = round(65536 p) of 65536 are dropped, m = 65536 / (65536 - n)
           for the others.  Sixteen bits decide: half column % 2 (low first) of word
           column / 2 % 4 of Philox4x32 in ten rounds (Salmon, Moraes, Dror, Shaw: Parallel Random
           Numbers: As Easy as 1, 2, 3, 2011), key = seed, counter = (column / 8, row, offset),
           the offset in 64 bits; below n the element is dropped.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def listed():
    return [
        # One new token in each of eight sequences through the packed projection of Q, K and V:
        # latency, and the weights read once.
        dict(name="linear_few_tokens", op="linear", step="fwd", T=8, K=768, N=2304, act="none", bias=True,
             residual=False, p=0.0, dtype="bf16"),
        # One token through a wide layer (32 heads of 128 columns): the weights' bytes bound it.
        dict(name="linear_one_token_wide", op="linear", step="fwd", T=1, K=4096, N=16384, act="silu", bias=False,
             residual=False, p=0.0, dtype="bf16"),
        # A training step of the same projection on eight sequences of 1024 tokens.
        dict(name="linear_gpt2s_qkv_step", op="linear", step="step", T=8192, K=768, N=2304, act="none", bias=True,
             residual=False, p=0.0, dtype="bf16"),
        # The way out of a feed-forward block of that model: dropout and the residual stream.
        dict(name="linear_gpt2s_out_step", op="linear", step="step", T=8192, K=2048, N=768, act="none", bias=True,
             residual=True, p=0.1, dtype="bf16"),
        # The way into it inside a Hessian-vector product.
        dict(name="linear_gpt2s_in_second", op="linear", step="second", T=8192, K=768, N=2048, act="gelu_tanh",
             bias=True, residual=False, p=0.0, dtype="bf16"),
        # A wide layer's training step (8192 tokens of the model of 32 heads of 128 columns).
        dict(name="linear_wide_step", op="linear", step="step", T=8192, K=4096, N=11008, act="silu", bias=False,
             residual=False, p=0.0, dtype="bf16"),
        # Sizes that are no multiples of anything, through the second order.
        dict(name="linear_odd_second", op="linear", step="second", T=1237, K=773, N=1531, act="gelu", bias=True,
             residual=True, p=0.2, dtype="bf16"),
        # A small model in 32 bits.
        dict(name="linear_fp32_step", op="linear", step="step", T=1021, K=512, N=2048, act="gelu", bias=True,
             residual=False, p=0.0, dtype="fp32"),
        # Dropout of one new token per sequence (a model sampled with its dropout on): latency.
        dict(name="dropout_few_rows", op="dropout", step="fwd", T=8, D=768, residual=True, p=0.1, dtype="bf16"),
        # A training step on the residual stream, eight sequences of 1024 tokens.
        dict(name="dropout_gpt2s_step", op="dropout", step="step", T=8192, D=768, residual=True, p=0.1, dtype="bf16"),
        # The same of a wide model, four sequences of 8192 tokens, forward.
        dict(name="dropout_wide_fwd", op="dropout", step="fwd", T=32768, D=4096, residual=False, p=0.5, dtype="bf16"),
        # Odd sizes in 32 bits.
        dict(name="dropout_odd_fp32", op="dropout", step="step", T=5003, D=1537, residual=True, p=0.25, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    p = rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.9), 3)])
    residual = rng.random() < 0.5
    if op == "dropout":
        D = rng.choice([_log(rng, 16, 16384), 8 * _log(rng, 8, 1024)])
        T = _log(rng, 1, max(1, min(65536, (2 ** 26) // D)))
        return dict(op=op, step=rng.choice(["fwd", "step"]), T=T, D=D, residual=residual, p=p, dtype=dtype)
    step = rng.choice(["fwd", "step", "second"])
    K = rng.choice([_log(rng, 16, 8192), 8 * _log(rng, 4, 1024)])
    N = rng.choice([_log(rng, 16, 16384), 8 * _log(rng, 4, 2048)])
    room = 2 ** (37 if dtype == "bf16" else 34) // (2 if step == "second" else 1)
    T = _log(rng, 1, max(1, min(16384, room // (K * N))))
    return dict(op=op, step=step, T=T, K=K, N=N, act=rng.choice(_ACTS), bias=rng.random() < 0.6, residual=residual,
                p=p, dtype=dtype)


# --- what a user's program holds -------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        x = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return x.mul_(std).to(dt)

    s = dict(case)
    # the generator's key, this call's place, and the training step's counter, which a captured
    # step keeps on the device
    s["seed"] = (int(seed) * 0x9E3779B97F4A7C15 + 12345) % 2 ** 63
    s["offset"] = 3 + int(seed) % 5 * 2 ** 31
    s["counter"] = torch.randint(0, 2 ** 40, (1,), generator=g, device="cuda")
    if own:  # the description of the dropout (no data), which a model keeps
        import exact_second_order_attn_gb300 as fb
        s["drop"] = fb.Dropout(case["p"], seed=s["seed"], offset=s["offset"])
    if case["op"] == "dropout":
        T, D = case["T"], case["D"]
        s["x"] = normal(T, D)
        s["r"] = normal(T, D) if case["residual"] else None
        if case["step"] == "step":
            s["dy"] = normal(T, D, std=0.1)
        return s
    T, K, N = case["T"], case["K"], case["N"]
    s["x"], s["W"] = normal(T, K), normal(N, K, std=1.0 / math.sqrt(K))
    s["b"] = normal(N, std=0.2) if case["bias"] else None
    s["r"] = normal(T, N) if case["residual"] else None
    if case["step"] != "fwd":
        s["dy"] = normal(T, N, std=0.1)
    if case["step"] == "second":
        s["ux"], s["uW"] = normal(T, K), normal(N, K, std=1.0 / math.sqrt(K))
        s["ub"] = normal(N) if case["bias"] else None
    return s


# --- plain forms --------------------------------------------------------------------------------

_LOW = 0xFFFFFFFF


def _factor(s, rows, cols):
    """m [rows, cols], or None without dropout."""
    n = round(65536 * s["p"])
    if n == 0:
        return None
    dev = s["counter"].device
    place = s["counter"] + s["offset"]
    c = [torch.arange((cols + 7) // 8, device=dev)[None, :], torch.arange(rows, device=dev)[:, None],
         place & _LOW, (place >> 32) & _LOW]
    k0, k1 = s["seed"] & _LOW, s["seed"] >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # modulo 2^64
        c = [((b >> 32) & _LOW) ^ c[1] ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c[3] ^ k1, a & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    bits = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], -1).reshape(rows, -1)[:, :cols]
    return (bits >= n).float() * (65536.0 / (65536 - n) if n < 65536 else 0.0)


def _activation(kind, z):
    """a(z), a'(z) and a''(z) (None where it vanishes)."""
    if kind == "none":
        return z, 1.0, None
    if kind == "relu":
        up = (z > 0).to(z.dtype)
        return z * up, up, None
    if kind == "silu":
        e = 1 / (1 + (-z).exp())
        d = e * (1 - e)
        return z * e, e + z * d, d * (2 + z * (1 - 2 * e))
    if kind == "gelu":
        up = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        bell = (-0.5 * z * z).exp() * (1 / math.sqrt(2 * math.pi))
        return z * up, up + z * bell, bell * (2 - z * z)
    # gelu_tanh: z (1 + tanh v) / 2 = z / (1 + exp(-2 v)), v = c (z + 0.044715 z^3)
    c = 2 * math.sqrt(2 / math.pi)
    w, w1, w2 = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z), c * 6 * 0.044715 * z
    e = 1 / (1 + (-w).exp())
    d = e * (1 - e)
    return z * e, e + z * d * w1, d * (2 * w1 + z * w2 + z * w1 * w1 * (1 - 2 * e))


def _plain_dropout(s):
    m = _factor(s, s["T"], s["D"])
    dt = s["x"].dtype
    y = s["x"].float() if m is None else s["x"].float() * m
    out = {"y": (y if s["r"] is None else y + s["r"].float()).to(dt)}
    if s["step"] == "step":
        out["dx"] = (s["dy"].float() if m is None else s["dy"].float() * m).to(dt)
    return out


def _plain_linear(s):
    dt = s["x"].dtype
    x, W = s["x"].float(), s["W"].float()
    z = x @ W.T
    if s["b"] is not None:
        z = z + s["b"].float()
    m = _factor(s, s["T"], s["N"])
    m = 1.0 if m is None else m
    a, a1, a2 = _activation(s["act"], z)
    y = a * m
    out = {"y": (y if s["r"] is None else y + s["r"].float()).to(dt)}
    if s["step"] == "fwd":
        return out
    dy = s["dy"].float() * m
    dz = dy * a1
    out["dx"], out["dW"] = (dz @ W).to(dt), (dz.T @ x).to(dt)
    if s["b"] is not None:
        out["db"] = dz.sum(0).to(dt)
    if s["step"] == "step":
        return out
    # vector-Jacobian product of (dx, dW, db) as functions of (x, W, b, dy)
    ux, uW = s["ux"].float(), s["uW"].float()
    t = ux @ W.T + x @ uW.T
    if s["b"] is not None:
        t = t + s["ub"].float()
    out["gdy"] = (m * t * a1).to(dt)
    gx, gW = dz @ uW, dz.T @ ux
    if a2 is not None:
        q = dy * t * a2
        gx, gW = gx + q @ W, gW + q.T @ x
        if s["b"] is not None:
            out["gb"] = q.sum(0).to(dt)
    elif s["b"] is not None:
        out["gb"] = torch.zeros_like(s["b"])
    out["gx"], out["gW"] = gx.to(dt), gW.to(dt)
    return out


# --- the framework's calls ----------------------------------------------------------------------

def _own_dropout(fb, s):
    out = {"y": fb.fbob_dropout_apply(s["drop"], s["x"], s["r"], counter=s["counter"])}
    if s["step"] == "step":
        out["dx"] = fb.fbob_dropout_apply(s["drop"], s["dy"], counter=s["counter"])
    return out


def _own_linear(fb, s):
    how = dict(activation=s["act"], dropout=s["drop"] if s["p"] > 0 else None,
               counter=s["counter"] if s["p"] > 0 else None)
    y, z = fb.fbob_linear_fwd(s["x"], s["W"], s["b"], s["r"], keep=s["step"] != "fwd", **how)
    out = {"y": y}
    if s["step"] != "fwd":
        want = (True, True, s["b"] is not None)
        out["dx"], out["dW"], db = fb.fbob_linear_bwd(s["x"], s["W"], z, s["dy"], want=want, **how)
        if s["b"] is not None:
            out["db"] = db
    if s["step"] == "second":
        want = (True, True, s["b"] is not None, True)
        out["gx"], out["gW"], gb, out["gdy"] = fb.fbob_linear_bob(s["x"], s["W"], z, s["dy"], s["ux"], s["uW"],
                                                                  s["ub"], want=want, **how)
        if s["b"] is not None:
            out["gb"] = gb
    return out


def run(state):
    if own:
        import exact_second_order_attn_gb300 as fb
        return (_own_linear if state["op"] == "linear" else _own_dropout)(fb, state)
    return (_plain_linear if state["op"] == "linear" else _plain_dropout)(state)


# --- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        n = case["T"] * case["D"]
        big = 2 + case["residual"] + (2 if case["step"] == "step" else 0)
        return dict(bytes=big * n * e, flops=2 * n * (2 if case["step"] == "step" else 1))
    T, K, N = case["T"], case["K"], case["N"]
    # each input and output once: x, W, r, y; dy, dx, dW; ux, uW, gx, gW, gdy; b, db, ub, gb
    x, w, y = {"fwd": (1, 1, 1), "step": (2, 2, 2), "second": (4, 4, 3)}[case["step"]]
    vec = {"fwd": 1, "step": 2, "second": 4}[case["step"]] * case["bias"]
    # products of 2 T K N: z; dx, dW; t (2), gx (2), gW (2), half of the last two without a''
    curved = case["act"] not in ("none", "relu")
    products = {"fwd": 1, "step": 3, "second": 9 if curved else 7}[case["step"]]
    return dict(bytes=(x * T * K + w * N * K + (y + case["residual"]) * T * N + vec * N) * e,
                flops=products * 2 * T * K * N)


# --- 64 bits --------------------------------------------------------------------------------------

def _exact_factor(case, s, rows, cols):
    n = int(round(65536 * case["p"]))
    if n == 0:
        return 1.0
    if n == 65536:
        return 0.0
    place = (int(s["counter"]) + s["offset"]) % 2 ** 64
    groups = (cols + 7) // 8
    keep = np.empty((rows, groups, 8), dtype=bool)
    for first in range(0, rows, 4096):
        some = np.arange(first, min(first + 4096, rows), dtype=np.uint64)[:, None]
        shape = (len(some), groups)
        x0 = np.broadcast_to(np.arange(groups, dtype=np.uint64)[None, :], shape)
        x1 = np.broadcast_to(some, shape)
        x2 = np.full(shape, place % 2 ** 32, dtype=np.uint64)
        x3 = np.full(shape, place // 2 ** 32, dtype=np.uint64)
        shift, low = np.uint64(32), np.uint64(2 ** 32 - 1)
        for i in range(10):
            key0 = np.uint64((s["seed"] + i * 0x9E3779B9) % 2 ** 32)
            key1 = np.uint64((s["seed"] // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)
            p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = (p1 >> shift) ^ x1 ^ key0, p1 & low, (p0 >> shift) ^ x3 ^ key1, p0 & low
        for j, word in enumerate((x0, x1, x2, x3)):
            keep[first:first + len(some), :, 2 * j] = word % np.uint64(65536) >= n
            keep[first:first + len(some), :, 2 * j + 1] = word // np.uint64(65536) >= n
    keep = torch.from_numpy(keep.reshape(rows, groups * 8)[:, :cols]).cuda()
    return keep.double() / (1.0 - n / 65536.0)


def _exact_act(kind, z):
    if kind == "relu":
        return torch.relu(z)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _exact_linear(case, s):
    first, second = case["step"] != "fwd", case["step"] == "second"
    m = _exact_factor(case, s, case["T"], case["N"])
    leaves = [s["x"], s["W"]] + ([s["b"]] if case["bias"] else [])
    leaves = [t.double().requires_grad_(first) for t in leaves]
    z = torch.nn.functional.linear(*leaves)
    y = _exact_act(case["act"], z) * m
    out = {"y": (y if s["r"] is None else y + s["r"].double()).detach()}
    if not first:
        return out
    dy = s["dy"].double().requires_grad_(second)
    got = torch.autograd.grad(y, leaves, dy, create_graph=second)
    out |= dict(zip(("dx", "dW", "db"), (t.detach() for t in got)))
    if second:
        u = [s[k].double() for k in ("ux", "uW", "ub")[:len(leaves)]]
        got = torch.autograd.grad(got, [dy] + leaves, u, allow_unused=True)
        got = [torch.zeros_like(l) if t is None else t for t, l in zip(got, [dy] + leaves)]
        out |= dict(zip(("gdy", "gx", "gW", "gb"), got))
    return out


def _exact_dropout(case, s):
    m = _exact_factor(case, s, case["T"], case["D"])
    y = s["x"].double() * m
    out = {"y": y if s["r"] is None else y + s["r"].double()}
    if case["step"] == "step":
        out["dx"] = s["dy"].double() * m
    return out


def exact(case, seed):
    if case["op"] == "linear" and work(case)["flops"] > 8e12:  # over about 20 s in 64 bits
        return None
    s = prepare(case, seed)
    return (_exact_linear if case["op"] == "linear" else _exact_dropout)(case, s)
