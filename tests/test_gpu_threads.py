"""Calls of the C ABI from two host threads at once (ctypes lets them run at
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


@pytest.mark.parametrize("few,many,D", [(1, 6000, 256), (1, 3000, 1024), (2, 2000, 2048)])
def test_layer_norm_of_few_and_of_many_rows(few, many, D):
    """One kernel serves both sizes, with different amounts of shared memory."""
    sides = [NormCalls(few, D, 1), NormCalls(many, D, 11)]
    torch.cuda.synchronize()
    for c in sides:
        assert c.run() == (_lib.OK,) * 3
    ref = [c.outputs() for c in sides]
    failed, start = [], threading.Barrier(2)

    def work(c):
        torch.cuda.set_device(0)
        start.wait()
        for i in range(ROUNDS):
            got = c.run()
            if got != (_lib.OK,) * 3:
                failed.append((c.desc.rows, i, got, c.lib.fbob_last_error().decode()))
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
