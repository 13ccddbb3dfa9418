"""A given stream has to be one of the tensors' device (no GPU: the check
precedes the call)."""

import types

import pytest
import torch

import exact_second_order_attn_gb300 as fb


def test_a_stream_of_another_device_is_refused():
    s = types.SimpleNamespace(device=torch.device("cuda", 1))
    x, y = torch.zeros(2, 3, 4, 8), torch.zeros(6, dtype=torch.int64)
    calls = (lambda: fb.fbob_rotary_apply(fb.Rotary(8), x, stream=s),
             lambda: fb.fbob_rotary_apply(fb.Rotary(8), x, x, stream=s),
             lambda: fb.fbob_layer_norm_fwd(x, stream=s),
             lambda: fb.fbob_linear_ce_fwd(x.view(6, 32), x.view(6, 32), y, stream=s))
    for call in calls:
        with pytest.raises(ValueError, match="stream"):
            call()
