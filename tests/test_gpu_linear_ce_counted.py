"""The linear head's cross entropy: the gradients of a few counted tokens are
as good among many ignored ones as alone."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from test_gpu_linear_ce import chain, compare, make

pytestmark = pytest.mark.gpu


def counted(t, got):
    """The problem and the results of the tokens that count."""
    rows = (t["target"] != -100).nonzero()[:, 0]
    tokens = ("H", "UH", "g", "target", "loss", "lse", "dH", "gH", "gg")
    return tuple({k: v[rows].contiguous() if k in tokens else v for k, v in d.items()} for d in (t, got))


@pytest.mark.parametrize("T,count,V,D", [(17, 16, 700, 64), (24, 4, 5003, 96), (300, 4, 1000, 64), (300, 16, 1000, 40),
                                         (65, 1, 129, 64), (5000, 2, 300, 32), (64, 3, 40007, 16), (1000, 15, 257, 768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_counted_tokens_among_ignored_ones(T, count, V, D, dtype):
    """Up to 16 counted tokens keep two bf16 terms of G and Z, whatever the
    number of rows: the bound is that of a batch of the counted tokens alone."""
    order = torch.randperm(T, generator=torch.Generator().manual_seed(T + count))
    t = make(T, D, V, dtype, seed=T + count, ignored=order[count:].tolist())
    got = chain(t)
    compare(*counted(t, got))
    for k in ("dH", "gH", "gg", "loss"):
        assert (got[k][order[count:].cuda()] == 0).all(), k


@pytest.mark.parametrize("T,count", [(300, 17), (300, 60), (64, 33)])
def test_more_counted_tokens(T, count):
    order = torch.randperm(T, generator=torch.Generator().manual_seed(T + count))
    t = make(T, 64, 900, "bf16", seed=count, ignored=order[count:].tolist())
    compare(*counted(t, chain(t)))


@pytest.mark.parametrize("piece", [256, 1024])
def test_few_counted_tokens_in_pieces(piece):
    order = torch.randperm(200, generator=torch.Generator().manual_seed(1))
    t = make(200, 64, 1500, "bf16", seed=3, ignored=order[5:].tolist())
    whole, cut = chain(t), chain(t, piece=piece)
    compare(*counted(t, cut))
    assert torch.equal(whole["dW"], cut["dW"]) and torch.equal(whole["gW"], cut["gW"])


@pytest.mark.parametrize("T", [16, 17, 500])
def test_a_replay_follows_the_count(T):
    """Captured with every token counted and replayed with three, and back."""
    t = make(T, 64, 600, "bf16", seed=T)
    full = t["target"].clone()
    few = torch.full_like(full, -100)
    few[2:5] = full[2:5]
    chain(t)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, lse = fb.fbob_linear_ce_fwd(t["H"], t["W"], t["target"])
        dH, dW = fb.fbob_linear_ce_bwd(t["H"], t["W"], t["target"], lse, t["g"])
        gH, gW, gg = fb.fbob_linear_ce_bob(t["H"], t["W"], t["target"], lse, t["g"], t["UH"], t["UW"])
    for y in (few, full, few):
        t["target"].copy_(y)
        g.replay()
        held = dict(loss=loss, lse=lse, dH=dH, dW=dW, gH=gH, gW=gW, gg=gg)
        for k, v in chain(t).items():
            assert torch.equal(v, held[k]), k
        compare(*counted(t, held))
