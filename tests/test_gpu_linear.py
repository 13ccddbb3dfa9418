"""Linear layers on the GPU: outputs, gradients and their vector-Jacobian
product against the fp64 oracle."""

import numpy as np
import pytest
import torch

import exact_second_order_attn_gb300 as fb
import oracle.model as om
from exact_second_order_attn_gb300 import _lib
from model_helpers import U32, check, draw, half_step, np64

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def make(T, K, N, dtype, seed=0, bias=True, residual=True):
    t = dict(x=draw(seed + 1, (T, K), dtype), W=draw(seed + 2, (N, K), dtype, K ** -0.5),
             dy=draw(seed + 3, (T, N), dtype), ux=draw(seed + 4, (T, K), dtype),
             uW=draw(seed + 5, (N, K), dtype, K ** -0.5), b=None, ub=None, r=None)
    if bias:
        t["b"], t["ub"] = draw(seed + 6, (N,), dtype, 0.3), draw(seed + 7, (N,), dtype)
    if residual:
        t["r"] = draw(seed + 8, (T, N), dtype)
    return t


def chain(t, act, drop=None, counter=None):
    how = dict(activation=act, dropout=drop, counter=counter)
    y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], **how)
    dx, dW, db = fb.fbob_linear_bwd(t["x"], t["W"], z, t["dy"], **how)
    gx, gW, gb, gdy = fb.fbob_linear_bob(t["x"], t["W"], z, t["dy"], t["ux"], t["uW"], t["ub"], **how)
    fb.device_status()
    return dict(y=y, z=z, dx=dx, dW=dW, db=db, gx=gx, gW=gW, gb=gb, gdy=gdy)


def compare(t, got, act, m):
    """Bounds, in magnitudes summed as the kernels sum them.

    z adds K products in fp32 (the tensor cores may drop the last bit of each of
    the K/16 steps; fp32 inputs also lose the products below 2^-24 of three-term
    operands): K/8 + 8 roundings of sum |x W| + |b| bound its error dz.  The
    kernels' activations are within `near` (1 + |z|) of the functions (2^-18 for
    bf16: 7.5e-8 of the normal integral, times z, and a few 2^-22 of 2^x and 1/x;
    2^-21 for fp32: a few roundings).  The gradients read z as it is kept (fp16
    beside bf16: half a step and 2^-25 absolute): a', a'' then move by 1.2 (the
    largest |a''| and |a'''| are 0.8 and 1.1) times what that is off, and relu's slope where z may change its sign.  dz and q are
    rounded to bf16 once for bf16 inputs, up to 16 tokens to two bf16 terms."""
    n = {k: 0.0 if v is None else np64(v) for k, v in t.items()}
    x, W, b, r, dy, ux, uW, ub = (n[k] for k in ("x", "W", "b", "r", "dy", "ux", "uW", "ub"))
    T, K = x.shape
    N = W.shape[0]
    bf = t["x"].dtype == torch.bfloat16
    h = half_step(t["x"].dtype)
    near = 2.0 ** (-18 if bf else -21)
    M = m if np.ndim(m) else np.full((T, N), float(m))
    steps = K / 8 + 8
    hz, tiny = (half_step(torch.float16), 2.0 ** -25) if bf else (h, 0.0)
    z = x @ W.T + b
    a, a1, a2 = om.activation(act, z)
    ez = steps * U32 * (np.abs(x) @ np.abs(W).T + np.abs(b))
    near = near * (1 + np.abs(z)) if act not in ("none", "relu") else 0.0
    check("y", got["y"], om.linear(x, W, b, r, act, m), M * np.abs(a) + np.abs(r), 4, extra=M * (1.2 * ez + near))
    if got["z"] is not None:
        check("z", got["z"], z, 0, 0, extra=ez + tiny)
    if act == "none":
        e1 = e2 = np.zeros_like(z)
    elif act == "relu":
        e1, e2 = (np.abs(z) <= 2 * ez + tiny) * 1.0, np.zeros_like(z)
    else:
        e1 = e2 = 1.2 * (1.01 * hz * np.abs(z) + ez + tiny) + near
    exact = act == "none" and not np.ndim(m)  # dz is dy itself
    q = 0.0 if exact else U32 if not bf else h if T > 16 else h ** 2
    g = M * np.abs(dy)
    dz = g * np.abs(a1)
    edz = g * e1 + 1.01 * q * (dz + g * e1) + 4 * U32 * dz
    sn, st = N / 8 + 64, T / 8 + 64  # roundings of the sums over outputs and tokens
    dx, dW, db = om.linear_bwd(x, W, b, dy, act, m)
    check("dx", got["dx"], dx, dz @ np.abs(W), sn, extra=edz @ np.abs(W))
    check("dW", got["dW"], dW, dz.T @ np.abs(x), st, extra=edz.T @ np.abs(x))
    if got["db"] is not None:
        check("db", got["db"], db, dz.sum(0), st, extra=(g * e1 + 4 * U32 * dz).sum(0))
    tt = np.abs(ux @ W.T + x @ uW.T + ub)
    et = 2 * steps * U32 * (np.abs(ux) @ np.abs(W).T + np.abs(x) @ np.abs(uW).T + np.abs(ub))
    gx, gW, gb, gdy = om.linear_bob(x, W, b, dy, ux, uW, ub, act, m)
    check("gdy", got["gdy"], gdy, M * tt * np.abs(a1), 4, extra=M * (et * (np.abs(a1) + e1) + tt * e1))
    Q = g * tt * np.abs(a2)
    eQ = g * (et * (np.abs(a2) + e2) + tt * e2)
    if act in ("none", "relu"):
        eQ = eQ * 0.0
    check("gb", got["gb"], gb, Q.sum(0), st, extra=(eQ + 6 * U32 * Q).sum(0))
    eQ = eQ + 1.01 * q * (Q + eQ) + 6 * U32 * Q
    check("gx", got["gx"], gx, Q @ np.abs(W) + dz @ np.abs(uW), 2 * sn, extra=eQ @ np.abs(W) + edz @ np.abs(uW))
    check("gW", got["gW"], gW, Q.T @ np.abs(x) + dz.T @ np.abs(ux), 2 * st, extra=eQ.T @ np.abs(x) + edz.T @ np.abs(ux))


SHAPES = [(1, 8, 8), (1, 1, 1), (2, 300, 5), (3, 64, 127), (8, 768, 300), (16, 520, 96), (17, 64, 40), (33, 7, 65),
          (128, 64, 128), (129, 72, 129), (255, 128, 255), (256, 256, 256), (257, 320, 264), (300, 768, 1000),
          (700, 40, 600), (20, 2056, 136), (513, 96, 24), (40, 1031, 515)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_against_oracle(T, K, N, dtype):
    act = ACTS[(T + K + N) % 5]
    t = make(T, K, N, dtype, seed=T + N)
    compare(t, chain(t, act), act, 1.0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", [(5, 40, 24), (40, 72, 136), (70, 33, 77)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_activations_with_dropout(act, T, K, N, dtype):
    """The mask is the generator's, with a counter on the device."""
    t = make(T, K, N, dtype, seed=3, residual=T != 40)
    drop = fb.Dropout(0.3, seed=2 ** 63 + 5, offset=2 ** 32 - 2)
    counter = torch.tensor([5], device="cuda")
    m = om.dropout_factor(T, N, 0.3, 2 ** 63 + 5, 2 ** 32 + 3)
    compare(t, chain(t, act, drop, counter), act, m)


@pytest.mark.parametrize("T", [4, 50])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_plain_products(T, dtype):
    """No bias, residual, activation or dropout: dz is dy itself."""
    t = make(T, 64, 88, dtype, seed=4, bias=False, residual=False)
    t["ub"] = None
    got = chain(t, "none")
    assert got["z"] is None
    compare(t, got, "none", 1.0)


def test_all_dropped_and_none_dropped():
    t = make(20, 32, 40, "bf16", seed=5)
    got = chain(t, "gelu", fb.Dropout(1.0))
    assert torch.equal(got["y"], t["r"]) and not any(got[k].any() for k in ("dx", "dW", "db", "gx", "gW", "gb", "gdy"))
    whole, got = chain(t, "gelu"), chain(t, "gelu", fb.Dropout(2.0 ** -18))  # rounds to none of 65,536
    for k in whole:
        assert torch.equal(whole[k], got[k])


@pytest.mark.parametrize("T", [6, 24])
def test_what_is_dropped_is_zero_whatever_stands_there(T):
    """Infinite and NaN values at dropped places leave no trace."""
    N = 64
    drop = fb.Dropout(0.5, seed=9)
    gone = torch.from_numpy(om.dropout_factor(T, N, 0.5, 9, 0) == 0).cuda()
    t = make(T, 16, N, "bf16", seed=6)
    want = chain(t, "silu", drop)
    t["dy"] = torch.where(gone, torch.tensor(float("nan"), device="cuda", dtype=torch.bfloat16), t["dy"])
    got = chain(t, "silu", drop)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    x = draw(7, (T, N), "bf16")
    bad = torch.where(gone, torch.full_like(x, float("inf")), x)
    assert torch.equal(fb.fbob_dropout_apply(drop, x), fb.fbob_dropout_apply(drop, bad))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,K,N", [(20000, 24, 40), (40, 20000, 24), (40, 24, 20000)])
def test_long_sums(T, K, N, dtype):
    """More than 16,384 terms of each contraction."""
    t = make(T, K, N, dtype, seed=8)
    compare(t, chain(t, "gelu_tanh"), "gelu_tanh", 1.0)


@pytest.mark.parametrize("T", [5, 60])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_each_output_alone(T, dtype):
    """Any subset of the outputs, any cotangent left out."""
    t = make(T, 72, 104, dtype, seed=10)
    for act, drop in (("none", None), ("relu", None), ("gelu", fb.Dropout(0.2, 3)), ("none", fb.Dropout(0.2, 3))):
        how = dict(activation=act, dropout=drop)
        whole = chain(t, act, drop)
        y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], keep=False, **how)
        assert z is None and torch.equal(y, whole["y"])
        for i, k in enumerate(("dx", "dW", "db")):
            got = fb.fbob_linear_bwd(t["x"], t["W"], whole["z"], t["dy"], want=[i == j for j in range(3)], **how)
            assert torch.equal(got[i], whole[k]) and sum(v is not None for v in got) == 1
        zero = {k: torch.zeros_like(t[k]) for k in ("ux", "uW", "ub")}
        for none in (("ux",), ("uW",), ("ub",), ("ux", "ub"), ("uW", "ub"), ()):
            u = [None if k in none else t[k] for k in ("ux", "uW", "ub")]
            full = [zero[k] if k in none else t[k] for k in ("ux", "uW", "ub")]
            ref = fb.fbob_linear_bob(t["x"], t["W"], whole["z"], t["dy"], *full, **how)
            got = fb.fbob_linear_bob(t["x"], t["W"], whole["z"], t["dy"], *u, **how)
            for a, b in zip(got, ref):
                assert torch.equal(a, b)
            for i in range(4):
                one = fb.fbob_linear_bob(t["x"], t["W"], whole["z"], t["dy"], *u, want=[i == j for j in range(4)], **how)
                assert torch.equal(one[i], got[i]) and sum(v is not None for v in one) == 1
    fb.device_status()


@pytest.mark.parametrize("T,K,N", [(9, 36, 50), (37, 65, 301), (37, 64, 300), (300, 130, 44), (260, 72, 136)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nothing_is_written_past_the_outputs(T, K, N, dtype):
    t = make(T, K, N, dtype, seed=11)
    ref = chain(t, "silu")
    sizes = dict(y=(T, N), z=(T, N), dx=(T, K), dW=(N, K), db=(N,), gx=(T, K), gW=(N, K), gb=(N,), gdy=(T, N))
    for shift in (0, 1):  # on 16 bytes and one element past them
        flat = {k: torch.full((int(np.prod(s)) + 64 + shift,), 9.0, dtype=ref[k].dtype, device="cuda")
                for k, s in sizes.items()}
        o = {k: flat[k][shift:shift + int(np.prod(s))].view(s) for k, s in sizes.items()}
        fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "silu", y=o["y"], z=o["z"])
        fb.fbob_linear_bwd(t["x"], t["W"], o["z"], t["dy"], "silu", dx=o["dx"], dW=o["dW"], db=o["db"])
        fb.fbob_linear_bob(t["x"], t["W"], o["z"], t["dy"], t["ux"], t["uW"], t["ub"], "silu", gx=o["gx"], gW=o["gW"],
                           gb=o["gb"], gdy=o["gdy"])
        for k in sizes:
            assert torch.equal(o[k], ref[k]), k
            assert (flat[k][-64:] == 9.0).all() and (flat[k][:shift] == 9.0).all(), k


@pytest.mark.parametrize("odd", ["dx", "dW"])
def test_one_gradient_off_its_bound(odd):
    """Results of one launch that leave by bulk stores and row by row."""
    T, K, N = 4000, 264, 520
    t = make(T, K, N, "bf16", seed=18)
    ref = chain(t, "gelu")
    flat = torch.empty(max(T, N) * K + 1, dtype=torch.bfloat16, device="cuda")
    out = {"dx": None, "dW": None, odd: flat[1:(T if odd == "dx" else N) * K + 1].view(-1, K)}
    for _ in range(5):
        flat.fill_(9.0)
        dx, dW, _ = fb.fbob_linear_bwd(t["x"], t["W"], ref["z"], t["dy"], "gelu", dx=out["dx"], dW=out["dW"])
        assert torch.equal(dx, ref["dx"]) and torch.equal(dW, ref["dW"])


def test_leading_dimensions_and_no_tokens():
    t = make(24, 40, 56, "bf16", seed=12)
    y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "gelu")
    y3, z3 = fb.fbob_linear_fwd(t["x"].view(2, 3, 4, 40), t["W"], t["b"], t["r"].view(2, 3, 4, 56), "gelu")
    assert y3.shape == (2, 3, 4, 56) and torch.equal(y3.view(24, 56), y) and torch.equal(z3.view(24, 56), z)
    e, ey = t["x"][:0], t["dy"][:0]
    y, z = fb.fbob_linear_fwd(e, t["W"], t["b"], None, "gelu")
    dx, dW, db = fb.fbob_linear_bwd(e, t["W"], z, ey, "gelu")
    gx, gW, gb, gdy = fb.fbob_linear_bob(e, t["W"], z, ey, e, t["uW"], t["ub"], "gelu")
    assert y.shape == (0, 56) and dx.shape == gx.shape == (0, 40) and gdy.shape == (0, 56)
    assert not any(v.any() for v in (dW, db, gW, gb))


def test_infinite_and_nan_inputs_reach_their_rows_only():
    for dtype, T in (("bf16", 4), ("bf16", 40), ("fp32", 4), ("fp32", 40)):
        t = make(T, 48, 56, dtype, seed=13)
        clean = chain(t, "gelu")
        t["x"][1, 3] = float("inf")
        t["x"][2, 5] = float("nan")
        y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "gelu")
        rows = [i for i in range(T) if i not in (1, 2)]
        assert torch.equal(y[rows], clean["y"][rows]) and torch.equal(z[rows], clean["z"][rows])
        assert torch.isnan(z[2]).all()
        dx, dW, db = fb.fbob_linear_bwd(t["x"], t["W"], z, t["dy"], "gelu")
        assert torch.isnan(dx[2]).all() and torch.equal(dx[rows], clean["dx"][rows]) and torch.isnan(db).all()
        # (among the terms of fp32 operands an infinite value meets zeros and both signs)
        assert torch.isnan(y[2]).all() and not torch.isfinite(y[1]).all()
        assert dtype == "fp32" or torch.isinf(y[1]).any()


@pytest.mark.parametrize("T", [8, 300])
def test_captured_calls_read_the_counter_when_they_run(T):
    """Two graphs over one workspace each, replayed with the counter moved on."""
    t = make(T, 72, 136, "bf16", seed=14)
    drop = fb.Dropout(0.25, seed=21, offset=100)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    chain(t, "gelu", drop, counter)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(t, "gelu", drop, counter)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    how = dict(activation="gelu", dropout=drop, counter=counter)
    with torch.cuda.graph(graph):
        y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], **how)
        first = fb.fbob_linear_bwd(t["x"], t["W"], z, t["dy"], **how)
        second = fb.fbob_linear_bob(t["x"], t["W"], z, t["dy"], t["ux"], t["uW"], t["ub"], **how)
        counter += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        ref = chain(t, "gelu", fb.Dropout(0.25, seed=21, offset=100 + step))
        got = dict(zip(("y", "z", "dx", "dW", "db", "gx", "gW", "gb", "gdy"), (y, z, *first, *second)))
        for k in got:
            assert torch.equal(got[k], ref[k]), k
    assert int(counter) == 3


def test_another_stream():
    t = make(100, 264, 520, "bf16", seed=15)
    ref = chain(t, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, z = fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "silu", stream=s)
    out = fb.fbob_linear_bwd(t["x"], t["W"], z, t["dy"], "silu", stream=s)
    s.synchronize()
    for got, k in zip((y, z, *out), ("y", "z", "dx", "dW", "db")):
        assert torch.equal(got, ref[k])


def test_the_same_bits_every_time():
    for dtype in ("bf16", "fp32"):
        t = make(1000, 264, 520, dtype, seed=16)
        ref = chain(t, "gelu")
        for _ in range(3):
            got = chain(t, "gelu")
            for k in ref:
                assert torch.equal(ref[k], got[k])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_withheld_stages_time_out(dtype):
    """The waits of the product kernels run out, the kernels return, and the
    context stays usable."""
    t = make(300, 264, 520, dtype, seed=17)
    ref = chain(t, "gelu")
    old = fb.fbob_set_wait_limit_ns(20_000_000)
    fb.fbob_debug_stall_producer(True)
    try:
        for call in (lambda: fb.fbob_linear_fwd(t["x"], t["W"], t["b"], t["r"], "gelu"),
                     lambda: fb.fbob_linear_bwd(t["x"], t["W"], ref["z"], t["dy"], "gelu"),
                     lambda: fb.fbob_linear_bob(t["x"], t["W"], ref["z"], t["dy"], t["ux"], t["uW"], t["ub"], "gelu")):
            call()
            with pytest.raises(fb.FbobError) as err:
                fb.device_status()
            assert err.value.status == _lib.ERR_TIMEOUT
    finally:
        fb.fbob_debug_stall_producer(False)
        fb.fbob_set_wait_limit_ns(old)
    got = chain(t, "gelu")
    for k in ref:
        assert torch.equal(ref[k], got[k])


def test_calls_from_several_host_threads():
    """Through the C ABI at the same time, each thread on its own stream and
    workspace: every call succeeds and computes what it computes alone."""
    import ctypes
    import threading
    lib = _lib.load()
    drop = fb.Dropout(0.25, 7, 8)

    def calls(dtype, T, K, N, act, seed):
        t = make(T, K, N, dtype, seed)
        ref = chain(t, act, drop)
        code = _lib.BF16 if dtype == "bf16" else _lib.FP32
        l = _lib.Linear(T, K, N, code, _lib.ACTIVATIONS[act])
        d, q = ctypes.byref(l), ctypes.byref(drop)
        ws = [torch.empty(lib.fbob_linear_workspace_bytes(d, q, i) + 16, dtype=torch.uint8, device="cuda") for i in range(3)]
        out = {k: torch.empty_like(v) for k, v in ref.items()}
        p = {k: ctypes.c_void_p(v.data_ptr()) for k, v in {**{k: v for k, v in t.items() if v is not None}, **out}.items()}
        p = {**{k: None for k in t}, **p}
        stream = torch.cuda.Stream()
        s = ctypes.c_void_p(stream.cuda_stream)

        def run():
            w = [(ctypes.c_void_p(v.data_ptr()), v.numel(), s) for v in ws]
            st = (lib.fbob_linear_fwd(d, q, None, *(p[k] for k in ("x", "W", "b", "r", "y", "z")), *w[0]),
                  lib.fbob_linear_bwd(d, q, None, *(p[k] for k in ("x", "W", "z", "dy", "dx", "dW", "db")), *w[1]),
                  lib.fbob_linear_bob(d, q, None, *(p[k] for k in ("x", "W", "z", "dy", "ux", "uW", "ub", "gx", "gW", "gb",
                                                                   "gdy")), *w[2]))
            assert st == (0, 0, 0)
        return run, stream, out, ref, (t, ws)

    jobs = [calls("bf16", 300, 264, 520, "gelu", 1), calls("fp32", 70, 72, 136, "silu", 2),
            calls("bf16", 8, 96, 64, "relu", 3), calls("bf16", 41, 33, 77, "gelu_tanh", 4)]
    torch.cuda.synchronize()
    failed = []

    def work(run):
        try:
            for _ in range(300):
                run()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j[0],)) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    fb.device_status()
    assert not failed
    for _, _, out, ref, _ in jobs:
        for k in ref:
            assert torch.equal(out[k], ref[k]), k
