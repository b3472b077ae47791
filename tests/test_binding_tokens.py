"""What the binding of the tokens' way to their experts and back refuses, on the CPU."""
import pytest
import torch

import moe_layer_align_amd as moe

X, ROWS = torch.zeros(6, 32, dtype=torch.bfloat16), torch.zeros(12, 32, dtype=torch.bfloat16)
POS = torch.zeros(6, 2, dtype=torch.int32)


def test_neither_gradient():
    with pytest.raises(ValueError, match="neither drows nor dweights"):
        moe.combine_grad(X, None, POS, out_dtype=None)


def test_the_weights_gradient_alone_is_checked_like_both():
    with pytest.raises(ValueError, match="GPU"):
        moe.combine_grad(X, ROWS, POS, out_dtype=None)
    with pytest.raises(ValueError, match="num_rows is 11"):
        moe.combine_grad(X, ROWS, POS, num_rows=11, out_dtype=None)
    with pytest.raises(TypeError, match="out_dtype must be a torch.dtype"):
        moe.combine_grad(X, ROWS, POS, out_dtype=0)
