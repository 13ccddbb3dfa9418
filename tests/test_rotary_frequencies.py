"""The rotary frequencies against 40 decimal digits: what their rounding makes
of an angle is below position * 2^-52 radians."""

import pytest

import exact_second_order_attn_gb300 as fb
from exact_second_order_attn_gb300.build import build

mp = pytest.importorskip("mpmath")


@pytest.mark.parametrize("rot", [2, 6, 24, 64, 96, 128, 256])
@pytest.mark.parametrize("base", [100.0, 10000.0, 500000.0])
@pytest.mark.parametrize("kind", ["none", "linear", "base", "parts"])
def test_frequencies(rot, base, kind):
    if kind == "base" and rot == 2:
        pytest.skip("scaling the base needs more than one pair")
    build()
    factor, original, slow, fast = 8.0, 8192.0, 1.0, 4.0
    got = fb.fbob_rotary_frequencies(fb.Rotary(rot, base=base, scaling=kind, factor=factor, original=original, slow=slow,
                                               fast=fast))
    with mp.workdps(40):
        b = mp.mpf(base)
        if kind == "base":
            b *= mp.mpf(factor) ** (mp.mpf(rot) / (rot - 2))
        for i, t in enumerate(got):
            want = b ** (-mp.mpf(2 * i) / rot)
            if kind == "linear":
                want /= factor
            if kind == "parts":
                w = min(max((original * want / (2 * mp.pi) - slow) / (fast - slow), 0), 1)
                want *= w + (1 - w) / factor
            assert abs(mp.mpf(t) - want) <= mp.mpf(2) ** -52
