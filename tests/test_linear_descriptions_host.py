"""What linear layers and dropout take as a description of a mask (no GPU)."""

import pytest
import torch

import exact_second_order_attn_gb300 as fb
from exact_second_order_attn_gb300.build import build


@pytest.mark.parametrize("other", [fb.Norm(4, 8, 0, 0, 1e-5), fb.Rotary(8), fb.LinearCe(1, 2, 3, 0, -100, 0), bytes(24), 0.1])
def test_other_descriptions_are_refused(other):
    """Norm has a Dropout's size: read as one it would be a p of 2e-323 and drop nothing."""
    build()
    x, W = torch.zeros(4, 8), torch.zeros(6, 8)
    for call in (lambda: fb.dropout(other, x), lambda: fb.fbob_dropout_apply(other, x),
                 lambda: fb.linear(x, W, dropout=other), lambda: fb.fbob_linear_fwd(x, W, dropout=other),
                 lambda: fb.fbob_linear_bwd(x, W, None, x, dropout=other),
                 lambda: fb.fbob_linear_bob(x, W, None, x, x, None, dropout=other)):
        with pytest.raises(TypeError, match="Dropout"):
            call()


def test_a_mask_is_needed_where_nothing_else_is_done():
    build()
    for call in (lambda: fb.dropout(None, torch.zeros(4, 8)), lambda: fb.fbob_dropout_apply(None, torch.zeros(4, 8))):
        with pytest.raises(TypeError, match="Dropout"):
            call()
