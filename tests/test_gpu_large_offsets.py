"""Element offsets past 32 bits: rows at the end of tensors of more than 2^31
elements, against the same rows computed alone."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb

pytestmark = pytest.mark.gpu


def filled(*shape, seed=1):
    x = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    flat, step = x.view(-1), 1 << 28
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.bfloat16))
    return x


def test_rotary_past_32_bits():
    B, H, N, d = 1, 33, 520_000, 128
    assert B * H * N * d > 2 ** 31
    r = fb.Rotary(64, interleaved=True)
    Q = filled(B, H, N, d)
    q = fb.fbob_rotary_apply(r, Q, offset=7)
    for n in (0, N // 2, N - 3):
        alone = fb.fbob_rotary_apply(r, Q[:, :, n:n + 3], offset=7 + n)
        assert torch.equal(q[:, :, n:n + 3], alone)


@pytest.mark.parametrize("D", [4096, 1537])
def test_layer_norm_past_32_bits(D):
    rows = 2 ** 31 // D + 1001
    x, w = filled(rows, D), filled(D, seed=2)
    y, mean, rstd = fb.fbob_layer_norm_fwd(x, w)
    dx, dw, _ = fb.fbob_layer_norm_bwd(x, w, mean, rstd, x)
    gx, _, gdy = fb.fbob_layer_norm_bob(x, w, mean, rstd, x, x)
    for a in (0, rows // 2 * 8 // 8, rows - 16):
        part = x[a:a + 16].clone()
        py, pm, pr = fb.fbob_layer_norm_fwd(part, w)
        pdx = fb.fbob_layer_norm_bwd(part, w, pm, pr, part)[0]
        pgx, _, pgdy = fb.fbob_layer_norm_bob(part, w, pm, pr, part, part)
        # the same row off another 16-byte bound is summed in another order
        for got, ref in ((y, py), (dx, pdx), (gx, pgx), (gdy, pgdy)):
            got = got[a:a + 16].float()
            assert (got - ref.float()).abs().max() <= 2 ** -7 * ref.float().abs().max()
    fb.device_status()


def test_linear_ce_past_32_bits():
    T, D, V = 2 ** 31 // 512 + 3001, 512, 300
    H, W = filled(T, D), filled(V, D, seed=3) * 0.05
    y = torch.randint(0, V, (T,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    g = torch.full((T,), 0.5, device="cuda")
    loss, lse = fb.fbob_linear_ce_fwd(H, W, y)
    dH, dW = fb.fbob_linear_ce_bwd(H, W, y, lse, g)
    fb.device_status()
    for a in (0, T // 2, T - 100):
        s = slice(a, a + 100)
        ploss, plse = fb.fbob_linear_ce_fwd(H[s].clone(), W, y[s].clone())
        pdH, _ = fb.fbob_linear_ce_bwd(H[s].clone(), W, y[s].clone(), plse, g[s].clone())
        assert torch.equal(loss[s], ploss) and torch.equal(lse[s], plse)
        # other slabs of the contraction: equal up to the last roundings
        assert (dH[s].float() - pdH.float()).abs().max() <= 2 ** -7 * pdH.float().abs().max()
    # dW from products of parts, in fp32
    ref = torch.zeros(V, D, device="cuda")
    for a in range(0, T, 1 << 18):
        s = slice(a, a + (1 << 18))
        p = torch.softmax(H[s].float() @ W.float().T, -1)
        p[torch.arange(len(p), device="cuda"), y[s]] -= 1
        ref += 0.5 * p.T @ H[s].float()
    # four million bf16-rounded terms of either sign
    assert (dW.float() - ref).norm() <= 5e-3 * ref.norm()
