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


class Meta(OnGpu):
    """A tensor of any size that has no memory."""

    def data_ptr(self):
        return 1 << 20


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(Meta)


HUGE = (1 << 32) + 8  # 8 in 32 bits


@pytest.mark.parametrize("name,call", [
    ("rows", lambda s, o: moe.grouped_gemm(meta(HUGE, 64), meta(3, 32, 64), o, meta(HUGE, 32), stream=s)),
    ("ids", lambda s, o: moe.grouped_gemm(meta(8, 64), meta(3, 32, 64), o, meta(8, 32), a_rows=meta(HUGE, dtype=I32),
                                          stream=s)),
    ("matrix rows", lambda s, o: moe.grouped_gemm(meta(HUGE, 64), meta(3, 32, 64), o, meta(8, 32),
                                                  a_rows=meta(8, dtype=I32), stream=s)),
    ("result rows", lambda s, o: moe.grouped_gemm(meta(8, 64), meta(3, 32, 64), o, meta(HUGE, 32),
                                                  out_rows=meta(8, dtype=I32), stream=s)),
    ("divisor", lambda s, o: moe.grouped_gemm(meta(8, 64), meta(3, 32, 64), o, meta(8, 32), a_rows=meta(8, dtype=I32),
                                              a_div=(1 << 32) + 1, stream=s)),
    ("negative divisor", lambda s, o: moe.grouped_gemm(meta(8, 64), meta(3, 32, 64), o, meta(8, 32),
                                                       a_rows=meta(8, dtype=I32), a_div=1 - (1 << 32), stream=s)),
    ("N", lambda s, o: moe.grouped_gemm(meta(8, 64), meta(3, HUGE, 64), o, meta(8, HUGE), stream=s)),
    ("K", lambda s, o: moe.grouped_gemm_dgrad(meta(8, 64), meta(3, 64, HUGE), o, meta(8, HUGE), stream=s)),
    ("4-bit N", lambda s, o: moe.grouped_gemm_w4(meta(8, 64), meta(3, HUGE, 32, dtype=torch.uint8),
                                                 meta(3, HUGE, 2, dtype=torch.uint8), o, meta(8, HUGE), stream=s)),
    ("dy rows", lambda s, o: moe.grouped_gemm_wgrad(meta(HUGE, 64), meta(HUGE, 32), o,
                                                    meta(3, 64, 32, dtype=torch.float32), stream=s)),
    ("dy width", lambda s, o: moe.grouped_gemm_wgrad(meta(8, HUGE), meta(8, 32), o,
                                                     meta(3, HUGE, 32, dtype=torch.float32), stream=s)),
    ("checkpoint rows", lambda s, o: moe.swiglu_checkpoint(
        meta(HUGE, 64), h=meta(HUGE, 32), codes=meta(HUGE, 64, dtype=torch.uint8),
        scales=meta(HUGE, 2, 1, dtype=torch.uint8), stream=s)),
    ("checkpoint width", lambda s, o: moe.swiglu_checkpoint(
        meta(8, 2 * HUGE), h=meta(8, HUGE), codes=meta(8, 2 * HUGE, dtype=torch.uint8),
        scales=meta(8, 2, HUGE // 32 + 1, dtype=torch.uint8), stream=s)),
    ("gradient rows", lambda s, o: moe.swiglu_checkpoint_grad(
        meta(HUGE, 64, dtype=torch.uint8), meta(HUGE, 2, 1, dtype=torch.uint8), meta(HUGE, 32), dgu=meta(HUGE, 64),
        h=meta(HUGE, 32), dweight=meta(HUGE, dtype=torch.float32), stream=s)),
])
def test_sizes_past_32_bits(calls, name, call):
    # the library's sizes are int32: a larger one must not become another size
    off = zeros(4, dtype=I32)
    with pytest.raises(ValueError, match="32 bits"):
        call(Stream(), off)
    assert not calls
