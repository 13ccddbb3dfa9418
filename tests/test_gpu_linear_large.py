"""Offsets past 2^31 elements in every matrix of a linear layer."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import U32

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -9  # half a step of bf16 where a value has just passed a power of two


def close(got, ref, size, halves=1.0):
    """Within the result's rounding, `halves` half steps of the sum of magnitudes `size`
    (operands that are rounded, and their errors) and 64 fp32 roundings of it."""
    assert ((got.double() - ref).abs() <= 2 * HALF * ref.abs() + (halves * HALF + 64 * U32) * size).all()


def test_tokens_times_outputs():
    """2^19 + 100 tokens of 4104 outputs: y and z, dx and dW through dz, gdy, q."""
    T, K, N = 2 ** 19 + 100, 16, 4104
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda").mul_(std).bfloat16()

    x, W, ux, uW = r(T, K), r(N, K, std=0.25), r(T, K), r(N, K, std=0.25)
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, 255, 256, 2 ** 18, T - 300, T - 2, T - 1], device="cuda")
    dy[rows] = r(len(rows), N)
    y, z = fb.fbob_linear_fwd(x, W, activation="silu")
    dx, dW, db = fb.fbob_linear_bwd(x, W, z, dy, "silu")
    gx, gW, gb, gdy = fb.fbob_linear_bob(x, W, z, dy, ux, uW, None, "silu")
    fb.device_status()
    X, Wd, U, Ud, G = (t.double() for t in (x[rows], W, ux[rows], uW, dy[rows]))
    Z = X @ Wd.T
    s = torch.sigmoid(Z)
    a1, a2 = s + Z * s * (1 - s), s * (1 - s) * (2 + Z * (1 - 2 * s))
    t = U @ Wd.T + X @ Ud.T
    # what a', a'' are off (z is kept in fp16: 2^-12 of it; the functions: 2^-18) and what t is
    # (64 roundings of the magnitudes in its sum), in units of the half steps below
    e = (1.2 * 2.0 ** -12 * Z.abs() + 2.0 ** -18 * (1 + Z.abs())) / HALF
    A1, A2 = a1.abs() + e, a2.abs() + e
    tm = t.abs() + 64 * U32 / HALF * (U.abs() @ Wd.abs().T + X.abs() @ Ud.abs().T)
    close(y[rows], Z * s, (Z * s).abs() + e)
    close(gdy[rows], t * a1, tm * A1)
    dz, q = G * a1, G * t * a2
    dzm, qm = G.abs() * A1, G.abs() * tm * A2
    close(dx[rows], dz @ Wd, dzm @ Wd.abs(), 2)
    close(dW, dz.T @ X, dzm.T @ X.abs(), 2)
    close(db, dz.sum(0), dzm.sum(0))
    close(gx[rows], q @ Wd + dz @ Ud, qm @ Wd.abs() + dzm @ Ud.abs(), 3)
    close(gW, q.T @ X + dz.T @ U, qm.T @ X.abs() + dzm.T @ U.abs(), 3)
    close(gb, q.sum(0), qm.sum(0), 2)
    assert not dx[1000:2000].any() and not gx[T - 2000:T - 1000].any()


@pytest.mark.parametrize("T", [1, 20])
def test_outputs_times_columns(T):
    """2^17 + 8 outputs of 2^14 + 8 columns."""
    K, N = 2 ** 14 + 8, 2 ** 17 + 8
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    W = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    n = torch.tensor([0, 7, 2 ** 16, N - 9, N - 1], device="cuda")
    W[n] = torch.randn(len(n), K, generator=g, device="cuda").bfloat16()
    y, _ = fb.fbob_linear_fwd(x, W)
    close(y[:, n], x.double() @ W[n].double().T, x.double().abs() @ W[n].double().abs().T)
    assert not y[:, 100:200].any()
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    dy[:, n] = torch.randn(T, len(n), generator=g, device="cuda").bfloat16()
    dx, dW, _ = fb.fbob_linear_bwd(x, W, None, dy, want=(True, True, False))
    fb.device_status()
    close(dx, dy[:, n].double() @ W[n].double(), dy[:, n].double().abs() @ W[n].double().abs())
    close(dW[n], dy[:, n].double().T @ x.double(), dy[:, n].double().abs().T @ x.double().abs())
    assert not dW[100:200].any()
