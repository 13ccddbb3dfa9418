"""How long a chain of the tensor cores gets in the gradients' long sums, by
the library's own functions: both products of the second order count."""

import pytest

from native_helpers import compiled


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return compiled(str(tmp_path_factory.mktemp("chains")), """
        #include "ce.h"
        extern "C" int chain(int nseg) { return fbob::ce::long_chain(nseg) * fbob::ce::kBK; }
        extern "C" int is_long(int K, int nseg) { return fbob::ce::long_sum(K, nseg); }
    """)


@pytest.mark.parametrize("nseg", [1, 2])
def test_chains_hold_16384_terms(host, nseg):
    assert host.chain(nseg) * nseg == 16384
    for K in (1, 64, 8192, 8193, 16384, 16385, 50257, 1 << 24):
        # a sum that keeps one chain has no more terms than a cut one's chain
        assert bool(host.is_long(K, nseg)) == (K * nseg > 16384)
