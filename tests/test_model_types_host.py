"""Types that the operators do not have are refused as types (no GPU)."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int32])
def test_unsupported_types(dtype):
    x = torch.zeros(3, 8)
    with pytest.raises(TypeError):
        fb.fbob_layer_norm_bwd(x, None, x[:, 0], x[:, 0], x, bias_dtype=dtype)
    with pytest.raises(TypeError):
        fb.norm_for(x, dtype)
    with pytest.raises(TypeError):
        fb.norm_for(x.to(dtype), torch.float32)
    with pytest.raises(TypeError):
        fb.linear_ce_for(x.to(dtype), x)
