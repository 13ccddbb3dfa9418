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
