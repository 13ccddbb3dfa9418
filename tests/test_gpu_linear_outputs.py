"""Outputs of linear layers at places, and with values, that other tests pass over."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import misaligned
from test_gpu_linear import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", ["y", "z"])
def test_results_that_leave_row_by_row_beside_a_residual_in_boxes(off):
    """y or z off 16 bytes, the residual on them, two tiles and more per block: the next
    residual's box is where the last y stood."""
    T, K, N = 256 * 160, 64, 264
    t = make(T, K, N, "bf16", seed=1)
    y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "silu")
    out = {"y": None, "z": None, off: misaligned({"y": y, "z": z}[off])}
    for _ in range(5):
        out[off].fill_(9.0)
        a, b = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "silu", **out)
        assert torch.equal(a, y) and torch.equal(b, z)
    fb.device_status()


@pytest.mark.parametrize("T", [5, 20, 40])
@pytest.mark.parametrize("N", [24, 21])
def test_an_infinite_direction_stays_with_the_tokens(T, N):
    """uW infinite at one place: t and q are infinite in that output's column and nowhere
    else, and their sum over the tokens is not touched by the rows past the last one."""
    K = 32
    t = make(T, K, N, "bf16", seed=T)
    t["x"], t["W"], t["dy"] = t["x"].abs() + 0.1, t["W"] * 0.01, t["dy"].abs() + 0.1  # a'' > 0 near 0
    t["b"].zero_()
    _, z = fb.fbob_linear_fwd(t["x"], t["W"], activation="silu")
    clean = fb.fbob_linear_bob(t["x"], t["W"], z, t["dy"], t["ux"], t["uW"], t["ub"], "silu")
    t["uW"][7, 3] = float("inf")
    got = fb.fbob_linear_bob(t["x"], t["W"], z, t["dy"], t["ux"], t["uW"], t["ub"], "silu")
    fb.device_status()
    others = [i for i in range(N) if i != 7]
    assert torch.isposinf(got[2][7]) and torch.equal(got[2][others], clean[2][others])  # gb
    assert torch.isposinf(got[3][:, 7]).all() and torch.equal(got[3][:, others], clean[3][:, others])  # gdy
