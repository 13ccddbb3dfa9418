"""Layer norm's column sums over tensors of more than 2^31 elements, against
the same sums in 64 bits."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from model_helpers import U32
from test_gpu_large_offsets import filled

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("D", [4096, 1537])
def test_column_sums_past_32_bits(D):
    """dy = x + v + 2 and ux = v with independent x and v: every term of dw, db
    and gw is near 1, 2 and 1 on average, so that left out or doubled rows show.

    Roundings: a thread adds up the rows of its block, at most rows / 304 in
    turn, then come 8 warps and 20 partial rows; a term itself carries at most
    300 of its row's magnitudes (as the tests of small sizes count them)."""
    rows = 2 ** 31 // D + 1001
    assert rows * D > 2 ** 31
    x, v = filled(rows, D), filled(rows, D, seed=2)
    dy = torch.empty_like(x)
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    step = 1 << 14
    for a in range(0, rows, step):
        s = slice(a, a + step)
        dy[s] = x[s].float() + v[s].float() + 2
    _, mean, rstd = fb.fbob_layer_norm_fwd(x, w, None, EPS)
    _, dw, db = fb.fbob_layer_norm_bwd(x, w, mean, rstd, dy, want=(False, True, True))
    _, gw, _ = fb.fbob_layer_norm_bob(x, w, mean, rstd, dy, v, want=(False, True, False))
    fb.device_status()
    ref = {k: torch.zeros(D, dtype=torch.float64, device="cuda") for k in ("dw", "db", "gw")}
    size = {k: r.clone() for k, r in ref.items()}
    rough = {k: r.clone() for k, r in ref.items()}
    for a in range(0, rows, step):
        s = slice(a, a + step)
        X, V, Y = (t[s].double() for t in (x, v, dy))
        X -= X.mean(-1, keepdim=True)
        r = ((X * X).mean(-1, keepdim=True) + EPS).rsqrt()
        xh = X * r
        pu = r * (V - V.mean(-1, keepdim=True) - xh * (V * xh).mean(-1, keepdim=True))
        big = xh.abs().amax(-1, keepdim=True) + 1  # the level of x is far below its spread
        pb = r * V.abs().amax(-1, keepdim=True) * (1 + big * big)
        for k, t, m in (("dw", Y * xh, Y.abs() * big), ("db", Y, 0 * Y), ("gw", pu * Y, Y.abs() * pb)):
            ref[k] += t.sum(0)
            size[k] += t.abs().sum(0)
            rough[k] += m.sum(0)
    for k, got in (("dw", dw), ("db", db), ("gw", gw)):
        bound = U32 * ((rows / 304 + 64) * size[k] + 300 * rough[k])
        assert got.dtype == torch.float32 and (got.double() - ref[k]).abs().le(bound).all(), k


@pytest.mark.parametrize("D", [4096, 1537])
def test_middle_rows_past_32_bits(D):
    """Rows from a multiple of 8 on, so that they lie on the same 16-byte bounds
    as alone: the same bits as a call on these rows."""
    rows = 2 ** 31 // D + 1001
    x, w = filled(rows, D), filled(D, seed=2)
    y, mean, rstd = fb.fbob_layer_norm_fwd(x, w)
    dx, _, _ = fb.fbob_layer_norm_bwd(x, w, mean, rstd, x, want=(True, False, False))
    gx, _, gdy = fb.fbob_layer_norm_bob(x, w, mean, rstd, x, x, want=(True, False, True))
    for a in (0, rows // 2 // 8 * 8, (rows - 16) // 8 * 8):
        part = x[a:a + 16].clone()
        py, pm, pr = fb.fbob_layer_norm_fwd(part, w)
        pdx = fb.fbob_layer_norm_bwd(part, w, pm, pr, part, want=(True, False, False))[0]
        pgx, _, pgdy = fb.fbob_layer_norm_bob(part, w, pm, pr, part, part, want=(True, False, True))
        for got, ref in ((y, py), (dx, pdx), (gx, pgx), (gdy, pgdy)):
            assert torch.equal(got[a:a + 16], ref)
    fb.device_status()
