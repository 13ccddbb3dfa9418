"""Shared helpers of the tests of the operators around the attention."""

from __future__ import annotations

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def draw(seed, shape, dtype="fp32", std=1.0, mean=0.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(TYPES.get(dtype, dtype)).to(device)


def np64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, ref, scale, terms, extra=0.0):
    """|got - ref| <= half a step of got's type relative to ref + ``terms``
    fp32 roundings of ``scale`` (the sum of the magnitudes that were added up)
    + ``extra`` (absolute, for roundings inside the kernel)."""
    ref = np.asarray(ref)
    x = np64(got)
    assert x.shape == ref.shape, f"{name}: {x.shape} != {ref.shape}"
    bound = half_step(got.dtype) * np.abs(ref) + (1 + half_step(got.dtype)) * (terms * U32 * scale + extra)
    off = np.abs(x - ref)
    assert np.isfinite(x).all(), f"{name}: not finite"
    worst = (off - bound).max() if off.size else -1.0
    assert worst <= 0.0, f"{name}: over the bound by {worst:.3g} (|ref| up to {np.abs(ref).max():.3g})"


def misaligned(t):
    """The same values one element past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    out = flat[1:].view(t.shape)
    out.copy_(t)
    return out
