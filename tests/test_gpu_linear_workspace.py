"""Linear layers with a workspace that holds NaN patterns, off a 256-byte bound."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from test_gpu_linear import compare, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,p", [("gelu", 0.0), ("silu", 0.3), ("relu", 0.0), ("none", 0.2), ("none", 0.0)])
@pytest.mark.parametrize("T,K,N", [(5, 40, 5), (16, 24, 127), (17, 33, 9), (40, 64, 301), (300, 72, 77), (70, 2056, 30)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nothing_is_read_that_was_not_written(dtype, T, K, N, act, p):
    """Whatever the workspace held (0xff bytes: NaN in every type, then zeros), and
    wherever it starts: the oracle's values, the same bits, nothing written around it."""
    t = make(T, K, N, dtype, seed=T + K + N)
    drop = fb.Dropout(p, seed=5, offset=6) if p else None
    how = dict(activation=act, dropout=drop)
    desc = fb.linear_for(t["x"], t["W"], act)

    def call(which, byte, start, f, *args):
        need = fb.fbob_linear_workspace_bytes(desc, which, drop)
        whole = torch.full((need + 1024,), 170, dtype=torch.uint8, device="cuda")
        first = -whole.data_ptr() % 256 + start
        whole[first:first + need] = byte
        out = f(*args, **how, workspace=whole[first:first + need])
        assert (whole[:first] == 170).all() and (whole[first + need:] == 170).all()
        return out

    def chain(byte, start):
        y, z = call(0, byte, start, fb.fbob_linear_fwd, t["x"], t["W"], t["b"], t["r"])
        dx, dW, db = call(1, byte, start, fb.fbob_linear_bwd, t["x"], t["W"], z, t["dy"])
        gx, gW, gb, gdy = call(2, byte, start, fb.fbob_linear_bob, t["x"], t["W"], z, t["dy"], t["ux"], t["uW"], t["ub"])
        fb.device_status()
        return dict(y=y, z=z, dx=dx, dW=dW, db=db, gx=gx, gW=gW, gb=gb, gdy=gdy)

    got = chain(255, 240)
    compare(t, got, act, om.dropout_factor(T, N, p, 5, 6) if p else 1.0)
    for k, v in chain(0, 16).items():
        assert v is None and got[k] is None or torch.equal(v, got[k]), k
