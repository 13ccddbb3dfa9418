"""Linear layers and dropout through autograd: alone, and together with the other
operators as a model uses them (norm -> projections -> rotary -> attention ->
projection with dropout and residual -> norm -> feed-forward block -> loss of a
linear head), gradients and Hessian-vector products through hvp()."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from model_helpers import U32, draw, misaligned

pytestmark = pytest.mark.gpu

B, N, H, d, V, F = 2, 37, 2, 32, 97, 120
D = H * d
DROPS = [fb.Dropout(0.2, seed=31, offset=i) for i in range(2)]
ACTS = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
        "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"), "silu": torch.nn.functional.silu}


def parameters(seed, dtype):
    g = torch.Generator().manual_seed(seed)

    def w(*shape, std, mean=0.0):
        return (torch.randn(*shape, generator=g, dtype=torch.float64) * std + mean).to(dtype).cuda()

    return [w(B * N, D, std=1.0), w(D, std=0.2, mean=1.0), w(D, std=0.2), w(3 * D, D, std=D ** -0.5), w(3 * D, std=0.1),
            w(D, D, std=D ** -0.5), w(D, std=0.1), w(D, std=0.2, mean=1.0), w(D, std=0.2), w(F, D, std=D ** -0.5),
            w(F, std=0.1), w(D, F, std=F ** -0.5), w(D, std=0.1), w(V, D, std=D ** -0.5)]


def targets():
    return torch.randint(0, V, (B * N,), generator=torch.Generator().manual_seed(5)).cuda()


def model(X, w1, b1, Wqkv, bqkv, Wo, bo, w2, b2, Wi, bi, Wd, bd, head):
    qkv = fb.linear(fb.layer_norm(X, w1, b1), Wqkv, bqkv).view(B, N, 3 * H, d)
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    q, k = fb.rotary(fb.Rotary(16), q, k)
    o = fb.attention(q, k, v.contiguous(), d ** -0.5, causal=True).to(X.dtype)
    X = fb.linear(o.transpose(1, 2).reshape(B * N, D), Wo, bo, residual=X, dropout=DROPS[0])
    h = fb.linear(fb.layer_norm(X, w2, b2), Wi, bi, activation="gelu")
    X = fb.dropout(DROPS[1], fb.linear(h, Wd, bd), X)
    return fb.linear_cross_entropy(X, head, targets()).mean()


def plain(X, w1, b1, Wqkv, bqkv, Wo, bo, w2, b2, Wi, bi, Wd, bd, head):
    """The same in torch's own double-precision operations."""
    def turn(x):
        i = torch.arange(8, device=x.device, dtype=x.dtype)
        a = torch.arange(N, device=x.device, dtype=x.dtype)[:, None] * 10000.0 ** (-2 * i / 16)
        p, q, rest = x[..., :8], x[..., 8:16], x[..., 16:]
        return torch.cat((p * a.cos() - q * a.sin(), p * a.sin() + q * a.cos(), rest), -1)

    m = [torch.from_numpy(om.dropout_factor(B * N, D, 0.2, 31, i)).cuda() for i in range(2)]
    qkv = (torch.nn.functional.layer_norm(X, (D,), w1, b1) @ Wqkv.T + bqkv).view(B, N, 3 * H, d)
    q, k, v = (qkv[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3))
    s = turn(q) @ turn(k).transpose(-1, -2) * d ** -0.5
    s = s.masked_fill(torch.ones(N, N, device=X.device, dtype=torch.bool).triu(1), float("-inf"))
    X = X + m[0] * ((s.softmax(-1) @ v).transpose(1, 2).reshape(B * N, D) @ Wo.T + bo)
    h = torch.nn.functional.gelu(torch.nn.functional.layer_norm(X, (D,), w2, b2) @ Wi.T + bi)
    X = X + m[1] * (h @ Wd.T + bd)
    return torch.nn.functional.cross_entropy(X @ head.T, targets())


def off(got, ref):
    return float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())


# Norms of differences.  fp32: some thirty steps of 2^-24 relative roundings on sums of
# up to a hundred terms, differentiated twice (each derivative multiplies by condition
# numbers of order ten): below 1e-4.  bf16: some twenty roundings of 2^-9 each, in
# quadrature 1 %, times the same factor: below 10 %.
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 0.1)])
def test_hessian_vector_product_of_a_block(dtype, tol):
    ps = [p.requires_grad_() for p in parameters(1, dtype)]
    vs = parameters(2, dtype)
    grads = torch.autograd.grad(model(*ps), ps)
    hv = fb.hvp(model, ps, vs)
    fb.device_status()
    qs = [p.detach().double().requires_grad_() for p in ps]
    first = torch.autograd.grad(plain(*qs), qs, create_graph=True)
    second = torch.autograd.grad(sum((g * v.double()).sum() for g, v in zip(first, vs)), qs)
    for i, (g, r) in enumerate(zip(grads, first)):
        assert off(g, r) < tol, i
    for i, (g, r) in enumerate(zip(hv, second)):
        assert off(g, r) < tol, i


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T", [3, 40])
def test_second_derivatives_of_any_subset(act, T):
    """fp32, every subset of (x, W, b, residual) that needs gradients: norms of
    differences below 30 roundings on sums of 40 terms."""
    K, M = 24, 32
    t = [draw(i, s, std=0.5) for i, s in enumerate(((T, K), (M, K), (M,), (T, M)))]
    gy = draw(9, (T, M))
    drop = fb.Dropout(0.25, 3, 4)
    m = torch.from_numpy(om.dropout_factor(T, M, 0.25, 3, 4)).cuda()
    for mask in range(1, 16):
        need = [bool(mask >> i & 1) for i in range(4)]
        a = [v.clone().requires_grad_(n) for v, n in zip(t, need)]
        e = [v.double().requires_grad_(n) for v, n in zip(t, need)]
        ya = fb.linear(a[0], a[1], a[2], residual=a[3], activation=act, dropout=drop)
        ye = m * ACTS[act](e[0] @ e[1].T + e[2]) + e[3]
        assert off(ya, ye) < 1e-6
        got, ref = [], []
        for y, leaves, out in ((ya, a, got), (ye, e, ref)):
            ls = [v for v, n in zip(leaves, need) if n]
            g = gy.to(y.dtype).requires_grad_()
            first = torch.autograd.grad(y, ls, g, create_graph=True)
            us = [draw(20 + i, v.shape).to(y.dtype) for i, v in enumerate(first)]
            second = torch.autograd.grad(first, [g] + ls, us, allow_unused=True)
            zero = [torch.zeros_like(v) if s is None else s for s, v in zip(second, [g] + ls)]
            out += [*first, *zero]
        for i, (g, r) in enumerate(zip(got, ref)):
            assert g.shape == r.shape and (off(g, r) < 2e-6 if r.abs().max() > 1e-12 else g.abs().max() < 1e-6), (mask, i)


def test_a_description_changed_after_the_forward():
    """The backward, and its own, draw by the description of their forward."""
    x, W, g = (draw(i, s).requires_grad_() for i, s in enumerate(((20, 16), (24, 16), (20, 24))))
    drop = fb.Dropout(0.5, 1, 2)
    want = fb.fbob_linear_bwd(x.detach(), W.detach(), None, g.detach(), dropout=drop, want=(True, False, False))[0]
    y = fb.linear(x, W, dropout=drop)
    drop.p, drop.seed = 0.1, 77
    (dx,) = torch.autograd.grad(y, x, g, create_graph=True)
    assert torch.equal(dx, want)
    u = draw(5, (20, 16))
    (gg,) = torch.autograd.grad(dx, g, u)
    again = fb.fbob_linear_bob(x.detach(), W.detach(), None, g.detach(), u, None, dropout=fb.Dropout(0.5, 1, 2),
                               want=(False, False, False, True))[3]
    assert torch.equal(gg, again)


def test_a_counter_that_moves_before_the_backward_is_noticed():
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    x = draw(1, (8, 16)).requires_grad_()
    y = fb.dropout(fb.Dropout(0.5), x, counter=counter)
    counter += 1
    with pytest.raises(RuntimeError, match="modified"):
        torch.autograd.grad(y.sum(), x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parameters_and_cotangents_that_are_views_of_one_vector(dtype):
    """Matrices that start on any element: the same bits (bf16 ones are copied).  fp32
    sums of few tokens are taken in another order: a term goes through 16 roundings at
    most (8 columns of a lane and their products, 5 steps over the lanes) each way."""
    T, K, M = 20, 64, 72

    def run(cut):
        ps = [draw(i, s, dtype) for i, s in enumerate(((T, K), (M, K), (M,), (T, M), (T, M)))]
        ps = [(misaligned(t) if cut else t).requires_grad_() for t in ps]
        y = fb.linear(*ps[:4], activation="gelu")
        first = torch.autograd.grad(y, ps[:3], ps[4], create_graph=True)
        us = [draw(10 + i, v.shape, dtype) for i, v in enumerate(first)]
        us = [misaligned(u) for u in us] if cut else us
        return [y, *first, *torch.autograd.grad(first, [*ps[:3], ps[4]], us)]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
    x, W = misaligned(draw(1, (4, K), dtype)), draw(2, (M, K), dtype)
    a, b = fb.linear(x, W), fb.linear(x.clone(), W)
    size = x.double().abs() @ W.double().abs().T
    limit = 0.0 if dtype == torch.bfloat16 else 32 * U32
    assert ((a.double() - b.double()).abs() <= limit * size).all()


def test_z_is_kept_only_for_gradients():
    x, W = draw(1, (30, 16)), draw(2, (24, 16)).requires_grad_()
    with torch.no_grad():
        y = fb.linear(x, W, activation="silu")
    assert y.grad_fn is None
    y = fb.linear(x, W.detach(), activation="silu", residual=draw(3, (30, 24)).requires_grad_())
    assert y.grad_fn.saved_tensors[3] is None
    y = fb.linear(x, W, activation="silu")
    assert y.grad_fn.saved_tensors[3] is not None
