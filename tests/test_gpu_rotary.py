"""Rotary positions on the GPU against the fp64 oracle."""

import numpy as np
import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from model_helpers import check, draw, misaligned, np64

pytestmark = pytest.mark.gpu

# An output is x0 c - x1 s (m <= 1.5 here) in fp32.  The angle is exact up to
# the rounding of its fraction of a half turn (half a step of at most 1, times
# pi), sincospif is good to 2 steps, m, the two products and the sum round
# once each: under 12 roundings of m (|x0| + |x1|).
TERMS = 12


def reference(x, pos, kw, transpose=False):
    kw = dict(kw)
    inter, m = kw.pop("interleaved", False), kw.pop("magnitude", 1.0)
    rot = kw.pop("rot")
    theta = om.rotary_theta(rot, **kw)
    y = om.rotary(np64(x), pos, theta, inter, m, transpose)
    mag = np.abs(np64(x))
    half = rot // 2
    scale = mag.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, half + i)
        scale[..., a] = scale[..., b] = abs(m) * (mag[..., a] + mag[..., b])
    return y, scale


CASES = [
    # B, H, Hk, N, d, rot
    (1, 1, 1, 1, 2, 2), (2, 3, 1, 5, 64, 64), (1, 2, 2, 129, 128, 64), (2, 4, 2, 33, 96, 96), (3, 1, 0, 17, 32, 16),
    (1, 5, 5, 70, 10, 6), (1, 1, 1, 9, 7, 4), (2, 2, 1, 31, 256, 256), (1, 3, 3, 40, 72, 24), (1, 33, 7, 6, 64, 48),
]


@pytest.mark.parametrize("shape", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary_against_oracle(shape, interleaved, dtype):
    B, H, Hk, N, d, rot = shape
    kw = dict(rot=rot, interleaved=interleaved, base=10000.0, scaling="parts", factor=4.0, original=512.0, slow=1.0,
              fast=8.0, magnitude=1.25)
    r = fb.Rotary(**kw)
    Q, K = draw(1, (B, H, N, d), dtype), draw(2, (B, Hk, N, d), dtype) if Hk else None
    pos = torch.arange(N)[None] * 3 - 4 + torch.arange(B)[:, None] * 100000
    for transpose in (False, True):
        out = fb.fbob_rotary_apply(r, Q, K, positions=pos.cuda(), transpose=transpose)
        out = out if K is not None else (out,)
        for name, x, y in zip("QK", (Q, K), out):
            ref, scale = reference(x, pos.numpy(), kw, transpose)
            check(name, y, ref, scale, TERMS)
            assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("kind", ["none", "linear", "base", "parts"])
def test_rotary_far_positions(kind):
    """Positions past 32 bits and below zero keep fp32 accuracy; int32, int64,
    shared and per-sequence positions and a plain offset agree."""
    kw = dict(rot=64, base=500000.0, scaling=kind, factor=8.0, original=8192.0)
    r = fb.Rotary(**kw)
    Q = draw(3, (2, 2, 6, 64))
    pos = torch.tensor([[0, 1, 2 ** 20 + 1, -5, 2 ** 31 - 1, 131071], [2 ** 33 + 7, -(2 ** 32), 77, 4, 3, 9]])
    # the oracle's own angle loses pos * 2^-53 * theta (below 1e-6 at 2^33): that much of |x| on top
    ref, scale = reference(Q, pos.numpy(), kw)
    check("int64", fb.fbob_rotary_apply(r, Q, positions=pos.cuda()), ref, scale, TERMS, extra=2e-6 * scale)
    small = torch.tensor([5, 0, 2 ** 31 - 1, -9, 44, 1 << 20], dtype=torch.int32)
    both = torch.stack([small, small])
    ref, scale = reference(Q, both.long().numpy(), kw)
    a = fb.fbob_rotary_apply(r, Q, positions=small.cuda())
    check("int32", a, ref, scale, TERMS, extra=1e-6 * scale)
    assert torch.equal(a, fb.fbob_rotary_apply(r, Q, positions=both.cuda()))
    assert torch.equal(a, fb.fbob_rotary_apply(r, Q, positions=(both - 1000).long().cuda(), offset=1000))
    seq = torch.arange(6)
    assert torch.equal(fb.fbob_rotary_apply(r, Q, offset=2 ** 40),
                       fb.fbob_rotary_apply(r, Q, positions=(seq + 2 ** 40).cuda()))
    assert torch.equal(fb.fbob_rotary_apply(r, Q), fb.fbob_rotary_apply(r, Q, positions=seq.cuda()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rotary_strides_alignment_and_outputs(dtype):
    """Packed views, rows off 16-byte boundaries and strided outputs give the
    contiguous call's results bit for bit; memory around them stays."""
    B, H, Hk, N, d = 2, 4, 2, 37, 64
    r = fb.Rotary(64)
    qkv = draw(4, (B, N, H + 2 * Hk, d), dtype)
    Q, K = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    ref = fb.fbob_rotary_apply(r, Q.contiguous(), K.contiguous())
    for a, b in zip(fb.fbob_rotary_apply(r, Q, K), ref):
        assert a.is_contiguous() and torch.equal(a, b)
    for a, b in zip(fb.fbob_rotary_apply(r, misaligned(Q.contiguous()), misaligned(K.contiguous())), ref):
        assert torch.equal(a, b)
    odd = torch.zeros(B, H, N, d + 1, dtype=Q.dtype, device="cuda")
    odd[..., :d] = Q
    assert torch.equal(fb.fbob_rotary_apply(r, odd[..., :d]), ref[0])
    out = torch.full((B, N, H + 2 * Hk, d), 7.0, dtype=Q.dtype, device="cuda")
    fb.fbob_rotary_apply(r, Q, K, Qo=out[:, :, :H].transpose(1, 2), Ko=out[:, :, H:H + Hk].transpose(1, 2))
    assert torch.equal(out[:, :, :H].transpose(1, 2), ref[0])
    assert torch.equal(out[:, :, H:H + Hk].transpose(1, 2), ref[1])
    assert (out[:, :, H + Hk:] == 7.0).all()
    # a query broadcast over the batch (stride 0) is read, never written
    one = Q[:1].expand(B, H, N, d)
    assert torch.equal(fb.fbob_rotary_apply(r, one)[1], fb.fbob_rotary_apply(r, Q[:1].contiguous())[0])


def test_rotary_special_values_stay_in_their_pair():
    """Infinities and NaN reach their own pair only; copied columns keep their bits."""
    r = fb.Rotary(8)
    x = draw(5, (1, 1, 3, 16))
    x[0, 0, 1, 2], x[0, 0, 1, 12], x[0, 0, 2, 15] = float("nan"), float("inf"), float("nan")
    y = fb.fbob_rotary_apply(r, x)
    bad = torch.isnan(y[0, 0])
    assert bad.nonzero().tolist() == [[1, 2], [1, 6], [2, 15]]
    assert y[0, 0, 1, 12] == float("inf")


def test_rotary_empty_and_many_heads():
    r = fb.Rotary(4)
    for shape in ((0, 2, 3, 8), (2, 0, 3, 8), (2, 2, 0, 8)):
        assert fb.fbob_rotary_apply(r, torch.empty(shape, device="cuda")).shape == shape
    x = draw(6, (1, 4000, 2, 8), "bf16")
    ref, scale = reference(x, np.array([[0, 1]]), dict(rot=4))
    check("many heads", fb.fbob_rotary_apply(r, x), ref, scale, TERMS)


def test_rotary_streams_and_graph():
    r = fb.Rotary(64, interleaved=True)
    Q, K = draw(7, (2, 4, 100, 64), "bf16"), draw(8, (2, 4, 100, 64), "bf16")
    ref = fb.fbob_rotary_apply(r, Q, K, offset=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = fb.fbob_rotary_apply(r, Q, K, offset=3, stream=s)
    with torch.cuda.stream(s):
        b = fb.fbob_rotary_apply(r, Q, K, offset=3)
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, ref):
        assert torch.equal(x, z) and torch.equal(y, z)
    pos = torch.arange(100, device="cuda") + 3
    qo, ko = torch.empty_like(Q), torch.empty_like(K)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fb.fbob_rotary_apply(r, Q, K, positions=pos, Qo=qo, Ko=ko)
    g.replay()
    assert torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])
    pos.add_(11)  # a replay reads the positions of its own time
    g.replay()
    assert torch.equal(qo, fb.fbob_rotary_apply(r, Q, K, offset=14)[0])


def test_rotary_gradients():
    """Backward, its double backward and partial use, against the transpose."""
    r = fb.Rotary(8, magnitude=1.5)
    Q, K = draw(9, (1, 2, 5, 12)).requires_grad_(), draw(10, (1, 1, 5, 12)).requires_grad_()
    q, k = fb.rotary(r, Q, K, offset=5)
    gq, gk = draw(11, q.shape).requires_grad_(), draw(12, k.shape)
    dQ, dK = torch.autograd.grad((q, k), (Q, K), (gq, gk), create_graph=True)
    tq, tk = fb.fbob_rotary_apply(r, gq.detach(), gk, offset=5, transpose=True)
    assert torch.equal(dQ, tq) and torch.equal(dK, tk)
    u = draw(13, Q.shape)
    (back,) = torch.autograd.grad(dQ, gq, u)
    assert torch.equal(back, fb.fbob_rotary_apply(r, u, offset=5))
    # differences of a linear map are exact up to rounding
    lhs, rhs = (np64(q) * np64(gq)).sum() + (np64(k) * np64(gk)).sum(), (np64(dQ) * np64(Q)).sum() + (np64(dK) * np64(K)).sum()
    assert lhs == pytest.approx(rhs, rel=1e-5)
    # K alone has a gradient; Q's is not asked for
    q, k = fb.rotary(r, Q.detach(), K, offset=5)
    (dK2,) = torch.autograd.grad(k.sum(), K)  # an expanded gradient
    assert torch.equal(dK2, fb.fbob_rotary_apply(r, torch.ones_like(k), offset=5, transpose=True))
    (dQ1,) = torch.autograd.grad(fb.rotary(r, Q, offset=5), Q, gq.detach())
    assert torch.equal(dQ1, tq)
