"""What the binding of the grouped products and the checkpointed activation
refuses or passes on, seen on the CPU: tensors that say they are on the GPU, and
a record in place of the library's call."""
import pytest
import torch

import moe_layer_align_amd as moe

BF16, I32 = torch.bfloat16, torch.int32


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on cuda:0; nothing follows its pointer."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class Stream:
    cuda_stream, device_index = 0x1000, 0


def gpu(t):
    return t.as_subclass(OnGpu)


def zeros(*shape, dtype=BF16):
    return gpu(torch.zeros(*shape, dtype=dtype))


@pytest.fixture
def calls(monkeypatch):
    out = []
    monkeypatch.setattr(moe._Call, "run", lambda self, fn, *args: out.append((fn, args)))
    return out


def struct(call):
    """The argument struct of a recorded call."""
    return call[1][0]._obj


def test_weight_gradient_wants_equal_rows(calls):
    # with the tokens' 6 rows in place of the 12 grouped ones (their ids forgotten), and the other way round
    off = zeros(4, dtype=I32)
    out = zeros(3, 16, 8, dtype=torch.float32)
    for n, m in ((12, 6), (6, 12), (1, 0), (0, 1)):
        with pytest.raises(ValueError, match="rows"):
            moe.grouped_gemm_wgrad(zeros(n, 16), zeros(m, 8), off, out, stream=Stream())
    assert not calls
    moe.grouped_gemm_wgrad(zeros(12, 16), zeros(12, 8), off, out, stream=Stream())
    assert struct(calls.pop()).R == 12
    # ids name the grouped rows of one operand; the other one holds at least as many, which the library checks
    ids = zeros(12, dtype=I32)
    moe.grouped_gemm_wgrad(zeros(12, 16), zeros(6, 8), off, out, a_rows=ids, a_div=2, stream=Stream())
    a = struct(calls.pop())
    assert (a.R, a.dy.rows, a.in_.rows, a.in_.div) == (12, 12, 6, 2)
    moe.grouped_gemm_wgrad(zeros(6, 16), zeros(15, 8), off, out, dy_rows=ids, dy_div=2, stream=Stream())
    a = struct(calls.pop())
    assert (a.R, a.dy.rows, a.in_.rows, a.dy.div) == (12, 6, 15, 2)
    with pytest.raises(ValueError):
        moe.grouped_gemm_wgrad(zeros(6, 16), zeros(6, 8), off, out, dy_rows=ids, a_rows=ids[:6], stream=Stream())
