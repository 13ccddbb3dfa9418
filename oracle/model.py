"""Plain fp64 NumPy oracle of the operators around the attention: rotary
positions, layer norm, the linear head's cross entropy, linear layers and
dropout, each with its first backward and that backward's vector-Jacobian product.  Test infrastructure
only; shares no code with the CUDA path.

The first backwards follow the chain rule node by node; the second-order
products come from differentiating each of those nodes (no closed row formula
is used, so the kernels' closed forms are checked against something else).
"""

from __future__ import annotations

import math

import numpy as np


# --- rotary positions -----------------------------------------------------------------------------

def rotary_theta(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, slow=1.0, fast=4.0):
    """theta_i as plain Python floats, i < rot/2."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        t = math.exp(-2.0 * i / rot * math.log(b))
        if scaling == "linear":
            t = t / factor
        if scaling == "parts":
            turns = original * t / (2.0 * math.pi)
            if turns <= slow:
                t = t / factor
            elif turns < fast:
                w = (turns - slow) / (fast - slow)
                t = w * t + (1.0 - w) * t / factor
        out.append(t)
    return out


def rotary(x, positions, theta, interleaved=False, magnitude=1.0, transpose=False):
    """x [B, H, N, d], positions [B, N] (integers); pair by pair."""
    y = np.array(x, dtype=np.float64)
    half = len(theta)
    for i, t in enumerate(theta):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        angle = np.asarray(positions, dtype=np.float64)[:, None, :] * t
        c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1.0 if transpose else 1.0)
        y[..., a] = c * x[..., a] - s * x[..., b]
        y[..., b] = s * x[..., a] + c * x[..., b]
    return y


# --- layer norm -----------------------------------------------------------------------------------

def layer_norm(x, w, b, eps):
    c = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return c * r * w + b


def layer_norm_bwd(x, w, dy, eps):
    """(dx, dw, db): reverse mode through c = x - mean, v = mean c^2, r = (v + eps)^-1/2, xh = c r."""
    D = x.shape[-1]
    c = x - x.mean(-1, keepdims=True)
    r = ((c * c).mean(-1, keepdims=True) + eps) ** -0.5
    a = dy * w                                  # adjoint of xh
    rb = (a * c).sum(-1, keepdims=True)         # of r
    vb = -0.5 * r ** 3 * rb                     # of v
    cb = a * r + 2.0 * c * vb / D               # of c
    dx = cb - cb.mean(-1, keepdims=True)
    return dx, (dy * c * r).sum(0), dy.sum(0)


def layer_norm_bob(x, w, dy, ux, uw, ub, eps):
    """(gx, gw, gdy): reverse mode through the nodes of layer_norm_bwd."""
    D = x.shape[-1]
    c = x - x.mean(-1, keepdims=True)
    r = ((c * c).mean(-1, keepdims=True) + eps) ** -0.5
    a = dy * w
    rb = (a * c).sum(-1, keepdims=True)
    vb = -0.5 * r ** 3 * rb
    # cotangents, from the outputs back
    t_cb = ux - ux.mean(-1, keepdims=True)      # dx = cb - mean cb
    t_dyxh = np.broadcast_to(uw, dy.shape)      # dw = sum dy c r
    t_a = t_cb * r
    t_r = (t_cb * a).sum(-1, keepdims=True) + (t_dyxh * dy * c).sum(-1, keepdims=True)
    t_c = 2.0 * t_cb * vb / D + t_dyxh * dy * r
    t_vb = (t_cb * 2.0 * c / D).sum(-1, keepdims=True)
    gdy = t_dyxh * c * r + ub
    t_r = t_r + t_vb * -1.5 * r ** 2 * rb       # vb = -0.5 r^3 rb
    t_rb = t_vb * -0.5 * r ** 3
    t_a = t_a + t_rb * c                        # rb = sum a c
    t_c = t_c + t_rb * a
    gdy = gdy + t_a * w                         # a = dy w
    gw = (t_a * dy).sum(0)
    t_v = t_r * -0.5 * r ** 3                   # r = (v + eps)^-1/2
    t_c = t_c + t_v * 2.0 * c / D
    gx = t_c - t_c.mean(-1, keepdims=True)
    return gx, gw, gdy


# --- cross entropy of a linear head -----------------------------------------------------------------

def _rows(target, ignore_index):
    return np.nonzero(target != ignore_index)[0]


def _whole(x, rows, T):
    out = np.zeros((T,) + x.shape[1:])
    out[rows] = x
    return out


def linear_ce(H, W, target, ignore_index=-100):
    """(loss, lse) per token; 0 where the target is ignored."""
    rows = _rows(target, ignore_index)
    z = H[rows] @ W.T
    top = z.max(-1) if len(rows) else np.zeros(0)
    lse = np.log(np.exp(z - top[:, None]).sum(-1)) + top
    return (_whole(lse - z[np.arange(len(rows)), target[rows]], rows, len(target)), _whole(lse, rows, len(target)))


def _probabilities(H, W, target, ignore_index):
    rows = _rows(target, ignore_index)
    h = H[rows]
    z = h @ W.T
    e = np.exp(z - z.max(-1, keepdims=True)) if len(rows) else z
    p = e / e.sum(-1, keepdims=True)
    one = np.zeros_like(p)
    one[np.arange(len(rows)), target[rows]] = 1.0
    return rows, h, p, one


def linear_ce_bwd(H, W, target, g, ignore_index=-100):
    """(dH, dW)."""
    rows, h, p, one = _probabilities(H, W, target, ignore_index)
    G = g[rows][:, None] * (p - one)
    return _whole(G @ W, rows, len(target)), G.T @ h


def linear_ce_bob(H, W, target, g, UH, UW, ignore_index=-100):
    """(gH, gW, gg): reverse mode through z = h W^T, p = softmax(z), q = p - one, G = g q, dH = G W, dW = G^T h."""
    rows, h, p, one = _probabilities(H, W, target, ignore_index)
    g_, uh = g[rows][:, None], UH[rows]
    q = p - one
    G = g_ * q
    t_G = uh @ W.T + h @ UW.T
    gW = G.T @ uh                       # dH = G W
    gh = G @ UW                         # dW = G^T h
    gg = (t_G * q).sum(-1)
    t_p = g_ * t_G
    t_z = p * (t_p - (p * t_p).sum(-1, keepdims=True))
    return _whole(gh + t_z @ W, rows, len(target)), gW + t_z.T @ h, _whole(gg, rows, len(target))


# --- linear layers and dropout ----------------------------------------------------------------------

def philox(c, key):
    """Four words of Philox4x32 in ten rounds as Python integers (Salmon, Moraes, Dror, Shaw: Parallel
    Random Numbers: As Easy as 1, 2, 3, 2011)."""
    c, (k0, k1) = list(c), key
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k0, q % 2 ** 32, (p >> 32) ^ c[3] ^ k1, p % 2 ** 32]
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return c


def dropout_factor(rows, cols, p, seed, offset):
    """m [rows, cols]: 0 where the element is dropped."""
    n = round(65536 * p)
    m = np.zeros((rows, cols))
    if n == 65536:
        return m
    for i in range(rows if n else 0):
        for g in range((cols + 7) // 8):
            words = philox([g, i, offset % 2 ** 32, offset // 2 ** 32], [seed % 2 ** 32, seed // 2 ** 32])
            for j in range(8 * g, min(8 * g + 8, cols)):
                m[i, j] = (words[j % 8 // 2] >> 16 * (j % 2)) % 65536 >= n
    return (m if n else m + 1) * (65536 / (65536 - n))


def activation(kind, z):
    """(a, a', a'') of each z."""
    if kind == "none":
        return z, np.ones_like(z), np.zeros_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0) * 1.0, np.zeros_like(z)
    if kind == "gelu":
        erfc = np.vectorize(math.erfc, otypes=[float])
        F, f = 0.5 * erfc(-z / math.sqrt(2)), np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * F, F + z * f, 2 * f - z * z * f
    if kind == "silu":
        v, v1, v2 = z / 2, 0.5, 0.0
    else:  # gelu_tanh
        k = math.sqrt(2 / math.pi)
        v, v1, v2 = k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z * z), k * 0.26829 * z
    t = np.tanh(v)  # a = z (1 + tanh v) / 2
    u = 1 - t * t
    return z * (1 + t) / 2, (1 + t + z * u * v1) / 2, u * v1 + z * (u * v2 - 2 * t * u * v1 * v1) / 2


def linear(x, W, b, r, kind, m):
    return r + m * activation(kind, x @ W.T + b)[0]


def linear_bwd(x, W, b, dy, kind, m):
    """(dx, dW, db)."""
    dz = m * dy * activation(kind, x @ W.T + b)[1]
    return dz @ W, dz.T @ x, dz.sum(0)


def linear_bob(x, W, b, dy, ux, uW, ub, kind, m):
    """(gx, gW, gb, gdy): reverse mode through z = x W^T + b, s = a'(z), dz = m dy s and the three products."""
    _, s, s1 = activation(kind, x @ W.T + b)
    dz = m * dy * s
    t_dz = ux @ W.T + x @ uW.T + ub
    gW = dz.T @ ux                      # dx = dz W
    gx = dz @ uW                        # dW = dz^T x
    gdy = t_dz * m * s
    t_z = t_dz * m * dy * s1
    return gx + t_z @ W, gW + t_z.T @ x, t_z.sum(0), gdy
