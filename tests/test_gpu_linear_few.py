"""Forwards of few tokens on both sides of the rule that chooses their kernel."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import TYPES, U32, half_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,T,K,N,tiles", [
    ("bf16", 1, 4096, 16384, False), ("bf16", 2, 4096, 16384, True), ("bf16", 4, 4096, 4096, False),
    ("bf16", 4, 4096, 4104, True), ("bf16", 16, 1024, 4096, False), ("bf16", 16, 1024, 4099, True),
    ("bf16", 16, 4096, 16384, True), ("bf16", 8, 4100, 4092, False), ("bf16", 8, 4100, 4096, True),
    ("bf16", 16, 20000, 1000, True), ("fp32", 16, 4096, 2048, False), ("fp32", 17, 512, 256, True)])
def test_the_kernel_of_few_tokens(dtype, T, K, N, tiles):
    """The tensor cores' tiles above 2^26 products of bf16 operands (2^27 where W is
    copied), and the same values either way: K/8 + 8 roundings of the sums of magnitudes
    (rows: K/8 products a lane at most and five steps over the lanes)."""
    g = torch.Generator(device="cuda").manual_seed(T + K)

    def r(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda").mul_(std).to(TYPES[dtype])

    x, W, b, res = r(T, K), r(N, K, std=K ** -0.5), r(N), r(T, N)
    fb.fbob_profile_report()
    fb.fbob_profile_enable(True)
    try:
        y, z = fb.fbob_linear_fwd(x, W, b, res, "relu", dropout=fb.Dropout(0.25, 3))
        fb.device_status()
    finally:
        fb.fbob_profile_enable(False)
    names = set(fb.fbob_profile_report())
    assert ("linear_rows" in names) != tiles and bool(names & {"linear_fwd", "linear_fwd_slabs"}) == tiles, names
    Z = x.double() @ W.double().T + b.double()
    size = x.double().abs() @ W.double().abs().T + b.double().abs()
    off = (K / 8 + 8) * U32 * size
    assert ((z.double() - Z).abs() <= half_step(z.dtype) * Z.abs() + 1.01 * (off + 2.0 ** -24)).all()
    m = fb.fbob_dropout_apply(fb.Dropout(0.25, 3), torch.ones(T, N, device="cuda")).double()
    Y = res.double() + m * Z.clamp(min=0)
    h = half_step(y.dtype)
    assert ((y.double() - Y).abs() <= h * Y.abs() + (1 + h) * (m * off + 4 * U32 * (m * Z.abs() + res.double().abs()))).all()
