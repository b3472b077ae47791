"""What the binding of the tokens' way to their experts and back refuses, on the CPU."""
import numpy as np
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


ID = torch.zeros(6, 2, dtype=torch.int32)
W = torch.zeros(6, 2)
CODES, CHANNELS = torch.zeros(4, 16, 32, dtype=torch.int8), torch.zeros(4, 16)
OFF = torch.zeros(5, dtype=torch.int32)


@pytest.mark.parametrize("n", [np.int64(4), np.int32(4), torch.tensor(4), True], ids=["int64", "int32", "tensor", "bool"])
@pytest.mark.parametrize("call", [
    lambda n: moe.dispatch(X, ID, n), lambda n: moe.dispatch(X, ID, 4, first_expert=n),
    lambda n: moe.combine_grad(X, None, POS, num_rows=n), lambda n: moe.route_topk_grad(ID, W, W, n),
    lambda n: moe.grouped_gemm_int8(X, CODES, CHANNELS, OFF, a_rows=OFF, a_div=n),
])
def test_integers_of_any_kind(call, n):
    # past the check of the argument, as in the functions that go through ctypes
    with pytest.raises(ValueError, match="GPU"):
        call(n)


@pytest.mark.parametrize("n", [4.0, np.float32(4), "4", None], ids=str)
def test_other_numbers_are_refused(n):
    with pytest.raises(TypeError, match="E must be an integer"):
        moe.dispatch(X, ID, n)


def test_integers_past_32_bits():
    for n in (np.int64(1 << 32), torch.tensor(1 << 32), 1 << 80):
        with pytest.raises(ValueError, match="32 bits"):
            moe.dispatch(X, ID, n)
    with pytest.raises(TypeError, match="integer"):
        moe.dispatch(X, ID, torch.tensor(4.0))
