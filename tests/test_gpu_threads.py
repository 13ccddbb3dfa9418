"""Calls of the C ABI from several host threads at once (ctypes lets them run at
the same time): every call succeeds and computes what it computes alone."""

import ctypes
import threading

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from exact_second_order_attn_gb300 import _lib
from model_helpers import draw

pytestmark = pytest.mark.gpu

ROUNDS = 1500


def p(t):
    return ctypes.c_void_p(t.data_ptr())


class NormCalls:
    """The three layer-norm passes on raw pointers, on a stream of their own."""

    def __init__(self, rows, D, seed):
        self.lib, self.stream = _lib.load(), torch.cuda.Stream()
        self.desc = _lib.Norm(rows, D, _lib.BF16, _lib.BF16, 1e-5)
        self.x, self.dy, self.ux = (draw(seed + i, (rows, D), "bf16") for i in range(3))
        self.w = draw(seed + 3, (D,), "bf16")
        self.big = [torch.empty_like(self.x) for _ in range(4)]      # y, dx, gx, gdy
        self.small = [torch.empty_like(self.w) for _ in range(3)]    # dw, db, gw
        self.mean, self.rstd = (torch.empty(rows, device="cuda") for _ in range(2))
        self.bytes = self.lib.fbob_layer_norm_workspace_bytes(ctypes.byref(self.desc))
        self.ws = torch.empty(self.bytes // 4, device="cuda")

    def run(self):
        """The statuses of one forward, backward and product of the backward."""
        d, s = ctypes.byref(self.desc), ctypes.c_void_p(self.stream.cuda_stream)
        y, dx, gx, gdy = map(p, self.big)
        dw, db, gw = map(p, self.small)
        x, w, dy, ux, mean, rstd = map(p, (self.x, self.w, self.dy, self.ux, self.mean, self.rstd))
        ws = (p(self.ws), self.bytes, s)
        return (self.lib.fbob_layer_norm_fwd(d, x, w, w, y, mean, rstd, s),
                self.lib.fbob_layer_norm_bwd(d, x, w, mean, rstd, dy, dx, dw, db, *ws),
                self.lib.fbob_layer_norm_bob(d, x, w, mean, rstd, dy, ux, w, w, gx, gw, gdy, *ws))

    def outputs(self):
        self.stream.synchronize()
        return [t.clone() for t in (*self.big, *self.small, self.mean, self.rstd)]


class HeadCalls:
    """The linear head's three passes, likewise."""

    def __init__(self, T, D, V, dtype, seed):
        self.lib, self.stream = _lib.load(), torch.cuda.Stream()
        self.desc = _lib.LinearCe(T, D, V, _lib.BF16 if dtype == "bf16" else _lib.FP32, -100, 0)
        self.H, self.UH = draw(seed, (T, D), dtype), draw(seed + 1, (T, D), dtype)
        self.W, self.UW = draw(seed + 2, (V, D), dtype, 0.2), draw(seed + 3, (V, D), dtype, 0.2)
        self.y = (torch.arange(T, device="cuda") * 7) % V
        self.g = draw(seed + 4, (T,))
        self.outs = [torch.empty_like(t) for t in (self.H, self.W, self.H, self.W, self.g, self.g, self.g)]
        self.bytes = [self.lib.fbob_linear_ce_workspace_bytes(ctypes.byref(self.desc), i) for i in range(3)]
        self.ws = torch.empty(max(self.bytes), dtype=torch.uint8, device="cuda")

    def run(self):
        d, s, ws = ctypes.byref(self.desc), ctypes.c_void_p(self.stream.cuda_stream), p(self.ws)
        H, W, y, g, UH, UW = map(p, (self.H, self.W, self.y, self.g, self.UH, self.UW))
        dH, dW, gH, gW, gg, loss, lse = map(p, self.outs)
        return (self.lib.fbob_linear_ce_fwd(d, H, W, y, loss, lse, ws, self.bytes[0], s),
                self.lib.fbob_linear_ce_bwd(d, H, W, y, lse, g, dH, dW, ws, self.bytes[1], s),
                self.lib.fbob_linear_ce_bob(d, H, W, y, lse, g, UH, UW, gH, gW, gg, ws, self.bytes[2], s))

    def outputs(self):
        self.stream.synchronize()
        return [t.clone() for t in self.outs]


class RotaryCalls:
    """One rotation of Q, each side by a description of its own."""

    def __init__(self, N, rot, seed):
        self.lib, self.stream = _lib.load(), torch.cuda.Stream()
        self.r = fb.Rotary(rot, base=100.0 * seed)
        self.x = draw(seed, (2, 3, N, 64), "bf16")
        self.y = torch.empty_like(self.x)
        self.heads = _lib.RotaryHeads(self.x.data_ptr(), self.y.data_ptr(), 3)
        self.heads.x_stride[:] = self.heads.y_stride[:] = (3 * N * 64, N * 64, 64)

    def run(self):
        s = ctypes.c_void_p(self.stream.cuda_stream)
        return (self.lib.fbob_rotary_apply(ctypes.byref(self.r), 2, self.x.shape[2], 64, _lib.BF16,
                                           ctypes.byref(self.heads), 1, None, 0, 0, 0, 0, s),) * 3

    def outputs(self):
        self.stream.synchronize()
        return [self.y.clone()]


def at_once(sides, rounds):
    torch.cuda.synchronize()
    for c in sides:
        assert c.run() == (_lib.OK,) * 3
    ref = [c.outputs() for c in sides]
    failed, start = [], threading.Barrier(len(sides))

    def work(c):
        torch.cuda.set_device(0)
        start.wait()
        for i in range(rounds):
            got = c.run()
            if got != (_lib.OK,) * 3:
                failed.append((type(c).__name__, i, got, c.lib.fbob_last_error().decode()))
                return
            if i % 100 == 99:
                c.stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for c, r in zip(sides, ref):
        for a, b in zip(c.outputs(), r):
            assert torch.equal(a, b)
    fb.device_status()


def test_heads_of_different_sizes_and_types():
    at_once([HeadCalls(5, 64, 700, "bf16", 1), HeadCalls(300, 96, 1500, "bf16", 11), HeadCalls(40, 64, 500, "fp32", 21)],
            300)


def test_rotations_by_different_descriptions():
    at_once([RotaryCalls(70, 64, 1), RotaryCalls(2000, 32, 2), RotaryCalls(1, 16, 3)], ROUNDS)


def test_all_operators():
    at_once([RotaryCalls(500, 64, 5), NormCalls(700, 768, 31), HeadCalls(60, 768, 900, "bf16", 41)], 300)


@pytest.mark.parametrize("few,many,D", [(1, 6000, 256), (1, 3000, 1024), (2, 2000, 2048)])
def test_layer_norm_of_few_and_of_many_rows(few, many, D):
    """One kernel serves both sizes, with different amounts of shared memory."""
    at_once([NormCalls(few, D, 1), NormCalls(many, D, 11)], ROUNDS)
