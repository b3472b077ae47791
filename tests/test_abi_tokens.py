"""Host-only checks of dispatch, combine, the router's gradient and the products
in 8-bit integers (no GPU needed): every refusal the header documents comes back
before anything is enqueued, and what the binding refuses or passes on."""
import ctypes

import pytest
import torch

import moe_layer_align_amd as moe
from test_abi_grouped import INVALID, OK, P, UNSUPPORTED, m, rows  # noqa: F401

BF16, F32, I32, I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
WORKSPACE = 3
VP, C32, C64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class DispatchArgs(ctypes.Structure):  # moe_dispatch_args_t
    _fields_ = [("M", C32), ("top_k", C32), ("E", C32), ("first_expert", C32), ("ids", VP), ("x", VP),
                ("x_stride", C64), ("row_bytes", C32), ("rows", VP), ("rows_stride", C64), ("offsets", VP),
                ("positions", VP), ("pairs", VP), ("workspace", VP), ("workspace_bytes", SZ)]


class CombineArgs(ctypes.Structure):  # moe_combine_args_t
    _fields_ = [("M", C32), ("top_k", C32), ("H", C32), ("R", C32), ("rows", VP), ("rows_stride", C64),
                ("rows_type", C32), ("positions", VP), ("weights", VP), ("y", VP), ("y_stride", C64), ("y_type", C32)]


class CombineGradArgs(ctypes.Structure):  # moe_combine_grad_args_t
    _fields_ = [("M", C32), ("top_k", C32), ("H", C32), ("R", C32), ("dy", VP), ("dy_stride", C64), ("dy_type", C32),
                ("rows", VP), ("rows_stride", C64), ("rows_type", C32), ("positions", VP), ("weights", VP),
                ("drows", VP), ("drows_stride", C64), ("drows_type", C32), ("dweights", VP)]


class GroupedInt8Args(ctypes.Structure):  # moe_grouped_int8_args_t
    _fields_ = [("R", C32), ("E", C32), ("N", C32), ("K", C32), ("offsets", VP), ("in_", moe._Rows), ("in_scale", VP),
                ("w", VP), ("w_scale", VP), ("out", moe._Rows), ("out_type", C32), ("workspace", VP),
                ("workspace_bytes", SZ)]


def call(m, name, cls, base, kw):  # noqa: F811
    d = dict(base)
    d.update(kw)
    f = getattr(m.load(), name)
    f.argtypes = [ctypes.POINTER(cls), VP]
    return f(ctypes.byref(cls(**d)), None)


def plain(m, name, *args):  # noqa: F811
    """A call without a struct: pointers, then sizes as the header has them."""
    kinds = {"moe_route_topk_grad": [VP, VP, VP, C32, C32, C32, VP, VP],
             "moe_quant_int8": [VP, C64, C32, C32, VP, VP, VP],
             "moe_swiglu_int8": [VP, C64, VP, C32, C32, VP, VP, VP, VP]}[name]
    f = getattr(m.load(), name)
    f.argtypes = kinds
    return f(*args)


DISPATCH = dict(M=10, top_k=2, E=4, first_expert=0, ids=P, x=P, x_stride=128, row_bytes=128, rows=P, rows_stride=128,
                offsets=P, positions=P, pairs=P, workspace=None, workspace_bytes=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(top_k=0), INVALID), (dict(first_expert=-1), INVALID),
    (dict(row_bytes=0), INVALID), (dict(x=None, rows=None, ids=None), INVALID),
    (dict(E=513), UNSUPPORTED), (dict(top_k=17), UNSUPPORTED),
    (dict(M=1 << 25), UNSUPPORTED), (dict(row_bytes=24, x_stride=32, rows_stride=32), UNSUPPORTED),
    (dict(row_bytes=1 << 22, x_stride=1 << 22, rows_stride=1 << 22), UNSUPPORTED),
    (dict(x_stride=1 << 22), UNSUPPORTED), (dict(rows_stride=1 << 22), UNSUPPORTED),
    (dict(ids=None), INVALID), (dict(ids=P + 2), INVALID), (dict(x=None), INVALID), (dict(x=P + 8), INVALID),
    (dict(rows=None), INVALID), (dict(rows=P + 4), INVALID), (dict(offsets=None), INVALID),
    (dict(offsets=P + 1), INVALID), (dict(positions=None), INVALID), (dict(positions=P + 2), INVALID),
    (dict(pairs=None), INVALID), (dict(pairs=P + 2), INVALID), (dict(x_stride=112), INVALID),
    (dict(x_stride=136), INVALID), (dict(rows_stride=112), INVALID), (dict(rows_stride=132), INVALID),
    (dict(M=2049), INVALID), (dict(M=2049, workspace=P + 8, workspace_bytes=1 << 20), INVALID),
    (dict(M=2049, workspace=P, workspace_bytes=95), WORKSPACE),
])
def test_dispatch_refusals(m, kw, code):  # noqa: F811
    assert call(m, "moe_dispatch", DispatchArgs, DISPATCH, kw) == code
    assert m.load().moe_dispatch(None, None) == INVALID


def test_dispatch_workspace(m):  # noqa: F811
    size = m.load().moe_dispatch_workspace_size
    assert size(2048, 2, 8) == 0 and size(2049, 2, 8) == (5 + 1) * 8 * 4
    assert size(-1, 2, 8) == size(5000, 0, 8) == size(5000, 2, 0) == size(5000, 2, 513) == size(1 << 25, 2, 8) == 0


COMBINE = dict(M=10, top_k=2, H=64, R=20, rows=P, rows_stride=64, rows_type=0, positions=P, weights=P, y=P, y_stride=64,
               y_type=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(R=-1), INVALID), (dict(top_k=0), INVALID), (dict(H=0), INVALID),
    (dict(rows_type=2), INVALID), (dict(y_type=-1), INVALID), (dict(H=60, rows_stride=64), UNSUPPORTED),
    (dict(top_k=17), UNSUPPORTED), (dict(M=1 << 25), UNSUPPORTED), (dict(R=(1 << 26) + 1), UNSUPPORTED),
    (dict(rows=None), INVALID), (dict(rows=P + 8), INVALID), (dict(rows_stride=56), INVALID),
    (dict(rows_stride=68), INVALID), (dict(rows_stride=1 << 21), UNSUPPORTED),
    (dict(rows_type=1, rows_stride=1 << 20), UNSUPPORTED), (dict(positions=None), INVALID),
    (dict(positions=P + 1), INVALID), (dict(weights=P + 2), INVALID), (dict(y=None), INVALID), (dict(y=P + 2), INVALID),
    (dict(y_stride=60), INVALID), (dict(y_stride=1 << 21), UNSUPPORTED),
])
def test_combine_refusals(m, kw, code):  # noqa: F811
    assert call(m, "moe_combine", CombineArgs, COMBINE, kw) == code
    assert m.load().moe_combine(None, None) == INVALID


GRAD = dict(M=10, top_k=2, H=64, R=20, dy=P, dy_stride=64, dy_type=0, rows=P, rows_stride=64, rows_type=0, positions=P,
            weights=P, drows=P, drows_stride=64, drows_type=0, dweights=P)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(R=-1), INVALID), (dict(top_k=-1), INVALID), (dict(H=-8), INVALID),
    (dict(dy_type=2), INVALID), (dict(rows_type=2), INVALID), (dict(drows_type=2), INVALID),
    (dict(H=12), UNSUPPORTED), (dict(top_k=17), UNSUPPORTED), (dict(M=1 << 25), UNSUPPORTED),
    (dict(R=(1 << 26) + 1), UNSUPPORTED), (dict(dy=None), INVALID), (dict(dy=P + 8), INVALID),
    (dict(dy_stride=56), INVALID), (dict(dy_stride=1 << 21), UNSUPPORTED), (dict(rows=None), INVALID),
    (dict(dweights=None), INVALID), (dict(rows=None, dweights=None, drows=None), INVALID),
    (dict(rows=P + 2), INVALID), (dict(rows_stride=62), INVALID), (dict(positions=None), INVALID),
    (dict(positions=P + 3), INVALID), (dict(weights=P + 2), INVALID), (dict(dweights=P + 2), INVALID),
    (dict(drows=P + 8), INVALID), (dict(drows_stride=0), INVALID), (dict(drows_stride=1 << 21), UNSUPPORTED),
])
def test_combine_grad_refusals(m, kw, code):  # noqa: F811
    assert call(m, "moe_combine_grad", CombineGradArgs, GRAD, kw) == code
    assert m.load().moe_combine_grad(None, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(E=513), UNSUPPORTED),
    (dict(k=17), UNSUPPORTED), (dict(M=1 << 25), UNSUPPORTED), (dict(ids=None), INVALID), (dict(w=None), INVALID),
    (dict(d=None), INVALID), (dict(out=None), INVALID), (dict(ids=P + 1), INVALID), (dict(w=P + 2), INVALID),
    (dict(d=P + 2), INVALID), (dict(out=P + 2), INVALID),
])
def test_route_grad_refusals(m, kw, code):  # noqa: F811
    d = dict(ids=P, w=P, d=P, M=4, E=8, k=2, out=P)
    d.update(kw)
    assert plain(m, "moe_route_topk_grad", d["ids"], d["w"], d["d"], d["M"], d["E"], d["k"], d["out"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(K=24), UNSUPPORTED), (dict(K=65552, stride=65552), UNSUPPORTED),
    (dict(M=1 << 26), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=P + 8), INVALID), (dict(stride=60), INVALID),
    (dict(stride=68), INVALID), (dict(stride=1 << 20), UNSUPPORTED), (dict(codes=None), INVALID),
    (dict(codes=P + 8), INVALID), (dict(scales=None), INVALID), (dict(scales=P + 2), INVALID),
])
def test_quant_refusals(m, kw, code):  # noqa: F811
    d = dict(x=P, stride=128, M=4, K=64, codes=P, scales=P)
    d.update(kw)
    assert plain(m, "moe_quant_int8", d["x"], d["stride"], d["M"], d["K"], d["codes"], d["scales"], None) == code
    if d["stride"] == 128:
        assert plain(m, "moe_swiglu_int8", d["x"], d["stride"], None, d["M"], d["K"], None, d["codes"], d["scales"],
                     None) == code


def test_swiglu_refusals(m):  # noqa: F811
    def f(*args):
        return plain(m, "moe_swiglu_int8", *args)

    assert f(P, 120, None, 4, 64, None, P, P, None) == INVALID  # a stride below 2 I
    assert f(P, 132, None, 4, 64, None, P, P, None) == INVALID
    assert f(P, 1 << 20, None, 4, 64, None, P, P, None) == UNSUPPORTED
    assert f(P, 128, P + 2, 4, 64, None, P, P, None) == INVALID
    assert f(P, 128, None, 4, 64, P + 1, P, P, None) == INVALID
    assert f(None, 0, None, 0, 64, None, None, None, None) == OK


def int8(m, in_=None, out=None, **kw):  # noqa: F811
    d = dict(R=10, E=4, N=64, K=128, offsets=P, in_scale=P, w=P, w_scale=P, out_type=0, workspace=None,
             workspace_bytes=0)
    d.update(kw)
    return call(m, "moe_grouped_gemm_int8", GroupedInt8Args, d,
                dict(in_=rows(m, d["K"], **(in_ or {})), out=rows(m, d["N"], **(out or {}))))


MANY = dict(R=1000, in_=dict(n=1000), out=dict(n=1000), in_scale=None, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-16), INVALID),
    (dict(out_type=2), INVALID), (dict(E=513), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(K=136), UNSUPPORTED),
    (dict(K=1 << 17), UNSUPPORTED), (dict(N=1 << 18, K=1 << 13), UNSUPPORTED), (dict(R=1 << 26), UNSUPPORTED),
    (dict(in_=dict(n=1 << 26, ids=P)), UNSUPPORTED), (dict(K=65552, in_scale=None), UNSUPPORTED),
    (dict(offsets=None), INVALID), (dict(offsets=P + 2), INVALID), (dict(w=None), INVALID), (dict(w=P + 8), INVALID),
    (dict(w_scale=None), INVALID), (dict(w_scale=P + 8), INVALID), (dict(in_scale=P + 2), INVALID),
    (dict(in_=dict(data=None)), INVALID), (dict(in_=dict(data=P + 8)), INVALID), (dict(in_=dict(stride=112)), INVALID),
    (dict(in_=dict(stride=136)), INVALID), (dict(in_=dict(stride=1 << 20)), UNSUPPORTED),
    (dict(in_=dict(n=9)), INVALID), (dict(in_=dict(div=2)), INVALID), (dict(in_=dict(ids=P, div=0)), INVALID),
    (dict(in_=dict(ids=P, n=(1 << 26) - 1)), UNSUPPORTED), (dict(out=dict(n=9)), INVALID),
    (dict(out=dict(data=P + 4)), INVALID), (dict(out=dict(ids=P, div=2)), INVALID),
    (dict(out=dict(stride=56)), INVALID),
    (dict(MANY, workspace=None), INVALID), (dict(MANY, workspace=P + 128), INVALID),
    (dict(MANY, workspace_bytes=1000 * 128 + 3999), WORKSPACE),
])
def test_product_refusals(m, kw, code):  # noqa: F811
    assert int8(m, **kw) == code
    assert m.load().moe_grouped_gemm_int8(None, None) == INVALID


def test_product_workspace(m):  # noqa: F811
    size = m.load().moe_grouped_int8_workspace_size
    assert size(1000, 4, 64, 128, 10) == 1280 + 40 and size(1000, 4, 64, 16, 3) == 256 + 12
    assert size(1000, 4, 64, 16, 0) == size(10, 4, 64, 128, 10) == 0  # the latter in one launch
    for bad in ((-1, 4, 64, 128, 9), (1000, 0, 64, 128, 9), (1000, 4, 0, 128, 9), (1000, 4, 64, 0, 9),
                (1000, 4, 64, 24, 9), (1000, 4, 64, 65552, 9), (1000, 4, 64, 128, -1), (1000, 4, 64, 128, 1 << 26)):
        assert size(*bad) == 0
    assert int8(m, R=0, offsets=None, w=None) == OK


def test_nothing_to_do(m):  # noqa: F811
    assert call(m, "moe_combine", CombineArgs, COMBINE, dict(M=0, rows=None, positions=None, y=None)) == OK
    assert call(m, "moe_combine_grad", CombineGradArgs, GRAD, dict(M=0, dy=None)) == OK
    assert plain(m, "moe_route_topk_grad", None, None, None, 0, 8, 2, None, None) == OK
    assert plain(m, "moe_quant_int8", None, 0, 0, 64, None, None, None) == OK


# ------------------------------------------------------------------ the binding
def zeros(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


IDS, OFF, W, WS = zeros(6, 2, dtype=I32), zeros(4, dtype=I32), zeros(3, 16, 32, dtype=I8), zeros(3, 16, dtype=F32)
P62 = zeros(6, 2, dtype=F32)  # weights of the pairs
ROWS, X = zeros(12, 32), zeros(6, 32)


@pytest.mark.parametrize("said,call", [
    ("out must have 32 columns and the rows", lambda: moe.dispatch(X, IDS, 4, zeros(11, 32))),
    ("out must not be Float", lambda: moe.dispatch(X, IDS, 4, zeros(12, 32, dtype=F32))),
    ("ids must be Int", lambda: moe.dispatch(X, IDS.long(), 4)),
    ("ids must be contiguous", lambda: moe.dispatch(X, zeros(2, 6, dtype=I32).t(), 4)),
    ("x must have 32 columns and the rows", lambda: moe.dispatch(X[:5], IDS, 4)),
    ("out needs x", lambda: moe.dispatch(None, IDS, 4, ROWS)),
    ("ids must be a tensor", lambda: moe.dispatch(X, None, 4)),
    ("ids must have shape", lambda: moe.dispatch(X, IDS[0], 4)),
    ("1, 2 or 4 bytes", lambda: moe.dispatch(X.double(), IDS, 4)),
    ("1, 2 or 4 bytes", lambda: moe.dispatch(X[0], IDS, 4)),
    ("x's rows must be contiguous", lambda: moe.dispatch(zeros(32, 6).t(), IDS, 4)),
    ("E must be an integer", lambda: moe.dispatch(X, IDS, 4.0)),
    ("weights must have shape", lambda: moe.combine(ROWS, IDS, zeros(6, 3, dtype=F32))),
    ("weights must be Float", lambda: moe.combine(ROWS, IDS, zeros(6, 2))),
    ("out must have 32 columns", lambda: moe.combine(ROWS, IDS, None, zeros(6, 24))),
    ("out must have 32 columns", lambda: moe.combine(ROWS, IDS, None, zeros(5, 32))),
    ("rows must not be Half", lambda: moe.combine(ROWS.half(), IDS)),
    ("out_dtype must be torch.bfloat16 or torch.float32", lambda: moe.combine(ROWS, IDS, out_dtype=torch.float16)),
    ("out_dtype must be a torch.dtype", lambda: moe.combine(ROWS, IDS, out_dtype="bf16")),
    ("rows must have 32 columns", lambda: moe.combine_grad(X, zeros(12, 24), IDS)),
    ("drows must have 32 columns", lambda: moe.combine_grad(X, ROWS, IDS, None, zeros(11, 32))),
    ("positions must have shape", lambda: moe.combine_grad(X[:5], ROWS, IDS)),
    ("dweights needs rows", lambda: moe.combine_grad(X, None, IDS, None, None, P62)),
    ("dweights must have shape", lambda: moe.combine_grad(X, ROWS, IDS, None, None, zeros(6, 3, dtype=F32))),
    ("num_rows is 11", lambda: moe.combine_grad(X, ROWS, IDS, num_rows=11)),
    ("num_rows is negative", lambda: moe.combine_grad(X, None, IDS, num_rows=-1)),
    ("dweights must have shape", lambda: moe.route_topk_grad(IDS, P62, zeros(6, 3, dtype=F32), 4)),
    ("out must have shape", lambda: moe.route_topk_grad(IDS, P62, P62, 4, zeros(6, 5, dtype=F32))),
    ("x must not be Float", lambda: moe.quant_int8(X.float())),
    ("codes must have shape", lambda: moe.quant_int8(X, zeros(6, 16, dtype=I8))),
    ("scales must be Float", lambda: moe.quant_int8(X, None, zeros(6))),
    ("gu must have shape", lambda: moe.swiglu_int8(zeros(4, 33))),
    ("num_rows must have shape", lambda: moe.swiglu_int8(X, num_rows=OFF)),
    ("row_weight must have shape", lambda: moe.swiglu_int8(X, zeros(5, dtype=F32))),
    ("int8 rows need a_scale", lambda: moe.grouped_gemm_int8(zeros(7, 32, dtype=I8), W, WS, OFF)),
    ("a_scale goes with int8 rows", lambda: moe.grouped_gemm_int8(X, W, WS, OFF, a_scale=zeros(6, dtype=F32))),
    ("a_scale must have shape", lambda: moe.grouped_gemm_int8(zeros(7, 32, dtype=I8), W, WS, OFF,
                                                              a_scale=zeros(8, dtype=F32))),
    ("w must be Char", lambda: moe.grouped_gemm_int8(X, W.view(torch.uint8), WS, OFF)),
    ("w_scale must have shape", lambda: moe.grouped_gemm_int8(X, W, zeros(3, 15, dtype=F32), OFF)),
    ("offsets must have shape", lambda: moe.grouped_gemm_int8(X, W, WS, OFF[:3])),
    ("input must have 32 columns", lambda: moe.grouped_gemm_int8(zeros(6, 48), W, WS, OFF)),
    ("the row ids must be Int", lambda: moe.grouped_gemm_int8(X, W, WS, OFF, a_rows=zeros(9))),
    ("the row ids must have shape", lambda: moe.grouped_gemm_int8(X, W, WS, OFF, zeros(6, 16), out_rows=OFF)),
    ("out must have 16 columns", lambda: moe.grouped_gemm_int8(X, W, WS, OFF, zeros(6, 24))),
    ("the weights must be a tensor", lambda: moe.grouped_gemm_int8(X, W[0], WS, OFF)),
])
def test_binding_refuses(said, call):
    with pytest.raises((TypeError, ValueError), match=said):
        call()


@pytest.mark.parametrize("call", [
    lambda: moe.dispatch(X, IDS, 4), lambda: moe.combine(ROWS, IDS, P62), lambda: moe.combine_grad(X, ROWS, IDS, P62),
    lambda: moe.route_topk_grad(IDS, P62, P62, 4), lambda: moe.quant_int8(X), lambda: moe.swiglu_int8(X),
    lambda: moe.grouped_gemm_int8(X, W, WS, OFF),
    lambda: moe.grouped_gemm_int8(zeros(6, 32, dtype=I8), W, WS, OFF, a_scale=zeros(6, dtype=F32), a_rows=IDS.view(-1)),
])
def test_binding_refuses_cpu_tensors(call):
    with pytest.raises(ValueError, match="GPU"):
        call()


HUGE = (1 << 32) + 8  # 8 in 32 bits


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


OFFM = meta(4, dtype=I32)


@pytest.mark.parametrize("name,call", [
    ("tokens", lambda: moe.dispatch(meta(HUGE, 64), meta(HUGE, 2, dtype=I32), 4, meta(2 * HUGE, 64))),
    ("pairs", lambda: moe.dispatch(meta(1 << 30, 64), meta(1 << 30, 4, dtype=I32), 4, meta(1 << 32, 64))),
    ("row bytes", lambda: moe.dispatch(meta(2, 1 << 31), meta(2, 2, dtype=I32), 4, meta(4, 1 << 31))),
    ("experts", lambda: moe.dispatch(meta(2, 64), meta(2, 2, dtype=I32), HUGE, meta(4, 64))),
    ("first", lambda: moe.dispatch(meta(2, 64), meta(2, 2, dtype=I32), 4, meta(4, 64), first_expert=HUGE)),
    ("rows", lambda: moe.combine(meta(HUGE, 64), meta(2, 2, dtype=I32), None, meta(2, 64))),
    ("combined", lambda: moe.combine(meta(2, 64), meta(HUGE, 2, dtype=I32), None, meta(HUGE, 64))),
    ("width", lambda: moe.combine(meta(2, HUGE), meta(2, 2, dtype=I32), None, meta(2, HUGE))),
    ("grad rows", lambda: moe.combine_grad(meta(2, 64), None, meta(2, 2, dtype=I32), None, meta(HUGE, 64),
                                                num_rows=HUGE)),
    ("logits", lambda: moe.route_topk_grad(meta(2, 2, dtype=I32), meta(2, 2, dtype=F32), meta(2, 2, dtype=F32),
                                                HUGE, meta(2, HUGE, dtype=F32))),
    ("quantised", lambda: moe.quant_int8(meta(HUGE, 64), meta(HUGE, 64, dtype=I8), meta(HUGE, dtype=F32))),
    ("activated", lambda: moe.swiglu_int8(meta(HUGE, 64), codes=meta(HUGE, 32, dtype=I8),
                                               scales=meta(HUGE, dtype=F32))),
    ("product rows", lambda: moe.grouped_gemm_int8(meta(HUGE, 64, dtype=I8), meta(3, 32, 64, dtype=I8),
                                                        meta(3, 32, dtype=F32), OFFM, meta(HUGE, 32),
                                                        a_scale=meta(HUGE, dtype=F32))),
    ("divisor", lambda: moe.grouped_gemm_int8(meta(8, 64, dtype=I8), meta(3, 32, 64, dtype=I8),
                                              meta(3, 32, dtype=F32), OFFM, meta(8, 32),
                                              a_scale=meta(8, dtype=F32), a_rows=meta(8, dtype=I32), a_div=HUGE)),
])
def test_sizes_past_32_bits(name, call):
    # the library's sizes are int32: a larger one must not become another size
    with pytest.raises(ValueError, match="32 bits"):
        call()
