"""The linear head's cross entropy with more columns than one chain of the
logits holds, over several tiles of tokens and of classes."""

import pytest

from test_gpu_linear_ce import chain, compare, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,V", [(300, 512, 700), (300, 520, 700), (520, 768, 515), (300, 1032, 300), (257, 2056, 600),
                                   (513, 4096, 257), (40, 8200, 130)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_wide_heads(T, D, V, dtype):
    t = make(T, D, V, dtype, seed=D, ignored=range(0, T, 7))
    compare(t, chain(t))
