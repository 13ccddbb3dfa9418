"""The linear head's calls with a workspace on any 16-byte bound."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from test_gpu_linear_ce import chain, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [16, 32, 48, 112, 240])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,V", [(33, 64, 300), (5, 12, 5003)])
def test_workspace_off_256_bytes(offset, dtype, T, D, V):
    """A workspace that starts `offset` bytes past a 256-byte bound, of exactly
    the size that was asked for: the same bits, and nothing written around it."""
    t = make(T, D, V, dtype, seed=offset, ignored=(1,))
    full = chain(t)
    a = (t["H"], t["W"], t["target"])
    calls = (lambda w: dict(zip(("loss", "lse"), fb.fbob_linear_ce_fwd(*a, workspace=w))),
             lambda w: dict(zip(("dH", "dW"), fb.fbob_linear_ce_bwd(*a, full["lse"], t["g"], workspace=w))),
             lambda w: dict(zip(("gH", "gW", "gg"), fb.fbob_linear_ce_bob(*a, full["lse"], t["g"], t["UH"], t["UW"],
                                                                         workspace=w))))
    for which, call in enumerate(calls):
        need = fb.fbob_linear_ce_workspace_bytes(fb.linear_ce_for(t["H"], t["W"]), which)
        guard = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
        start = -guard.data_ptr() % 256 + offset
        assert (guard.data_ptr() + start) % 256 == offset
        for k, v in call(guard[start:start + need]).items():
            assert torch.equal(v, full[k]), k
        assert (guard[:start] == 255).all() and (guard[start + need:] == 255).all()
    fb.device_status()
