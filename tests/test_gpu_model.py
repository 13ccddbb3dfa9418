"""The operators together, as a model around the attention uses them:
layer norm -> projections -> rotary -> attention -> projection -> layer norm ->
loss of a linear head, its gradients and Hessian-vector products through hvp()."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb

pytestmark = pytest.mark.gpu

B, N, H, d, V = 2, 37, 2, 32, 97
D = H * d
ROT = dict(rot=16, base=10000.0)


def parameters(seed, dtype):
    g = torch.Generator().manual_seed(seed)

    def w(*shape, std, mean=0.0):
        return (torch.randn(*shape, generator=g, dtype=torch.float64) * std + mean).to(dtype).cuda()

    return [w(B * N, D, std=1.0), w(D, std=0.2, mean=1.0), w(D, std=0.2), w(D, 3 * D, std=D ** -0.5),
            w(D, D, std=D ** -0.5), w(D, std=0.2, mean=1.0), w(D, std=0.2), w(V, D, std=D ** -0.5)]


def targets():
    y = torch.randint(0, V, (B * N,), generator=torch.Generator().manual_seed(5))
    y[::6] = -100
    return y.cuda()


def model(X, w1, b1, Wqkv, Wo, w2, b2, head):
    x = fb.layer_norm(X, w1, b1)
    qkv = (x @ Wqkv).view(B, N, 3 * H, d)
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    q, k = fb.rotary(fb.Rotary(**ROT), q, k)
    o = fb.attention(q, k, v.contiguous(), d ** -0.5, causal=True).to(X.dtype)
    X = X + o.transpose(1, 2).reshape(B * N, D) @ Wo
    loss = fb.linear_cross_entropy(fb.layer_norm(X, w2, b2), head, targets())
    return loss.sum() / (targets() != -100).sum()


def plain(X, w1, b1, Wqkv, Wo, w2, b2, head):
    """The same in torch's own double-precision operations."""
    def turn(x):
        i = torch.arange(ROT["rot"] // 2, device=x.device, dtype=x.dtype)
        a = torch.arange(N, device=x.device, dtype=x.dtype)[:, None] * ROT["base"] ** (-2 * i / ROT["rot"])
        p, q, rest = x[..., :8], x[..., 8:16], x[..., 16:]
        return torch.cat((p * a.cos() - q * a.sin(), p * a.sin() + q * a.cos(), rest), -1)

    x = torch.nn.functional.layer_norm(X, (D,), w1, b1)
    qkv = (x @ Wqkv).view(B, N, 3 * H, d)
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    s = turn(q) @ turn(k).transpose(-1, -2) * d ** -0.5
    s = s.masked_fill(torch.ones(N, N, device=x.device, dtype=torch.bool).triu(1), float("-inf"))
    X = X + (s.softmax(-1) @ v).transpose(1, 2).reshape(B * N, D) @ Wo
    z = torch.nn.functional.layer_norm(X, (D,), w2, b2) @ head.T
    return torch.nn.functional.cross_entropy(z, targets())


def off(got, ref):
    return float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())


# Norms of differences.  fp32: some twenty steps of 2^-24 relative roundings on
# sums of up to a hundred terms, differentiated twice (each derivative multiplies
# by condition numbers of order ten): below 1e-4.  bf16: a dozen roundings of
# 2^-9 each, in quadrature 1 %, times the same factor: below 10 %.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.1)])
def test_hessian_vector_product_of_a_block(dtype, tol):
    ps = [p.requires_grad_() for p in parameters(1, dtype)]
    vs = parameters(2, dtype)
    loss = model(*ps)
    grads = torch.autograd.grad(loss, ps)
    hv = fb.hvp(model, ps, vs)
    fb.device_status()
    qs = [p.detach().double().requires_grad_() for p in ps]
    ref = plain(*qs)
    first = torch.autograd.grad(ref, qs, create_graph=True)
    second = torch.autograd.grad(sum((a * v.double()).sum() for a, v in zip(first, vs)), qs)
    assert off(loss, ref) <= tol / 10
    for g, h, f, s in zip(grads, hv, first, second):
        assert g.dtype == h.dtype == dtype
        assert off(g, f) <= tol and off(h, s) <= tol


def test_a_training_step_captured_and_replayed():
    """Forward and backward through every operator in one CUDA graph: a replay
    on new values gives the eager step's gradients bit for bit."""
    values = parameters(3, torch.bfloat16)
    ps = [p.clone().requires_grad_() for p in values]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            torch.autograd.grad(model_static(*ps), ps)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = model_static(*ps)
        grads = torch.autograd.grad(loss, ps)
    for p, v in zip(ps, parameters(4, torch.bfloat16)):
        p.data.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    fresh = [p.detach().clone().requires_grad_() for p in ps]
    ref = model_static(*fresh)
    assert torch.equal(ref, loss)
    for a, b in zip(torch.autograd.grad(ref, fresh), grads):
        assert torch.equal(a, b)


_held = None


def model_static(*ps):
    """The model with targets made once (a captured step cannot copy from the host)."""
    global _held
    if _held is None:
        _held = targets()
    X, w1, b1, Wqkv, Wo, w2, b2, head = ps
    x = fb.layer_norm(X, w1, b1)
    qkv = (x @ Wqkv).view(B, N, 3 * H, d)
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    q, k = fb.rotary(fb.Rotary(**ROT), q, k)
    o = fb.attention(q, k, v.contiguous(), d ** -0.5, causal=True).to(X.dtype)
    X = X + o.transpose(1, 2).reshape(B * N, D) @ Wo
    return fb.linear_cross_entropy(fb.layer_norm(X, w2, b2), head, _held).mean()


def test_two_streams_at_once():
    """Calls in flight on two streams keep out of each other's way."""
    sets = [parameters(s, torch.bfloat16) for s in (6, 7)]
    y = targets()

    def work(ps):
        h, mean, rstd = fb.fbob_layer_norm_fwd(ps[0], ps[1], ps[2])
        loss, lse = fb.fbob_linear_ce_fwd(h, ps[7], y)
        dh, dW = fb.fbob_linear_ce_bwd(h, ps[7], y, lse, torch.ones_like(loss))
        return [loss, dh, dW, *fb.fbob_layer_norm_bwd(ps[0], ps[1], mean, rstd, dh)]

    ref = [work(ps) for ps in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (s, ps) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(work(ps))
    torch.cuda.synchronize()
    for r, rounds in zip(ref, got):
        for outs in rounds:
            for a, b in zip(outs, r):
                assert torch.equal(a, b)
