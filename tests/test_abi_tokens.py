"""Host-only checks of dispatch, combine, the router's gradient and the products
in 8-bit integers (no GPU needed): every refusal the header documents comes back
before anything is enqueued, and what the binding refuses or passes on."""
import ctypes

import pytest
import torch

import moe_layer_align_amd as moe
from test_abi_grouped import INVALID, OK, P, UNSUPPORTED, m, rows  # noqa: F401
from test_binding_grouped import HUGE, I32, Stream, calls, meta, struct, zeros  # noqa: F401

F32, I8 = torch.float32, torch.int8
WORKSPACE = 3


def call(m, name, cls, base, kw):  # noqa: F811
    d = dict(base)
    d.update(kw)
    return getattr(m.load(), name)(ctypes.byref(cls(**d)), None)


DISPATCH = dict(M=10, top_k=2, E=4, first_expert=0, ids=P, x=P, x_stride=128, row_bytes=128, rows=P, rows_stride=128,
                offsets=P, positions=P, pairs=P, workspace=None, workspace_bytes=0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(top_k=0), INVALID), (dict(first_expert=-1), INVALID),
    (dict(row_bytes=0), INVALID), (dict(E=513), UNSUPPORTED), (dict(top_k=17), UNSUPPORTED),
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
    assert call(m, "moe_dispatch", m._DispatchArgs, DISPATCH, kw) == code
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
    assert call(m, "moe_combine", m._CombineArgs, COMBINE, kw) == code
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
    assert call(m, "moe_combine_grad", m._CombineGradArgs, GRAD, kw) == code
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
    assert m.load().moe_route_topk_grad(d["ids"], d["w"], d["d"], d["M"], d["E"], d["k"], d["out"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(K=24), UNSUPPORTED), (dict(K=65552, stride=65552), UNSUPPORTED),
    (dict(M=1 << 26), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=P + 8), INVALID), (dict(stride=60), INVALID),
    (dict(stride=68), INVALID), (dict(stride=1 << 20), UNSUPPORTED), (dict(codes=None), INVALID),
    (dict(codes=P + 8), INVALID), (dict(scales=None), INVALID), (dict(scales=P + 2), INVALID),
])
def test_quant_refusals(m, kw, code):  # noqa: F811
    d = dict(x=P, stride=128, M=4, K=64, codes=P, scales=P)
    d.update(kw)
    assert m.load().moe_quant_int8(d["x"], d["stride"], d["M"], d["K"], d["codes"], d["scales"], None) == code
    if d["stride"] == 128:
        assert m.load().moe_swiglu_int8(d["x"], d["stride"], None, d["M"], d["K"], None, d["codes"], d["scales"],
                                        None) == code


def test_swiglu_refusals(m):  # noqa: F811
    f = m.load().moe_swiglu_int8
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
    a = m._GroupedInt8Args(in_=rows(m, d["K"], **(in_ or {})), out=rows(m, d["N"], **(out or {})), **d)
    return m.load().moe_grouped_gemm_int8(ctypes.byref(a), None)


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
    lib = m.load()
    assert call(m, "moe_combine", m._CombineArgs, COMBINE, dict(M=0, rows=None, positions=None, y=None)) == OK
    assert call(m, "moe_combine_grad", m._CombineGradArgs, GRAD, dict(M=0, dy=None)) == OK
    assert lib.moe_route_topk_grad(None, None, None, 0, 8, 2, None, None) == OK
    assert lib.moe_quant_int8(None, 0, 0, 64, None, None, None) == OK


# ------------------------------------------------------------------ the binding
def test_binding_passes_on(calls):  # noqa: F811
    # rows with a stride; types; what is made and how large
    s = Stream()
    x, ids = zeros(6, 48)[:, :32], zeros(6, 2, dtype=I32)
    moe.combine(zeros(12, 32, dtype=F32), ids, zeros(6, 2, dtype=F32), zeros(6, 32), stream=s)
    a = struct(calls.pop())
    assert (a.M, a.top_k, a.H, a.R, a.rows_type, a.y_type, a.rows_stride) == (6, 2, 32, 12, 1, 0, 32)
    moe.combine_grad(x, zeros(12, 32), ids, None, zeros(12, 32, dtype=F32), zeros(6, 2, dtype=F32), stream=s)
    a = struct(calls.pop())
    assert (a.dy_stride, a.dy_type, a.rows_type, a.drows_type, a.weights) == (48, 0, 0, 1, None)
    moe.combine_grad(x, None, ids, None, zeros(5, 32), num_rows=5, stream=s)
    a = struct(calls.pop())
    assert (a.R, a.rows, a.dweights) == (5, None, None)
    off, w, ws = zeros(4, dtype=I32), zeros(3, 16, 32, dtype=I8), zeros(3, 16, dtype=F32)
    moe.grouped_gemm_int8(zeros(7, 32, dtype=I8), w, ws, off, zeros(12, 16), a_scale=zeros(7, dtype=F32),
                          a_rows=zeros(12, dtype=I32), a_div=2, stream=s)
    a = struct(calls.pop())
    assert (a.R, a.E, a.N, a.K, a.in_.rows, a.in_.div, a.out_type, a.workspace) == (12, 3, 16, 32, 7, 2, 0, None)


@pytest.mark.parametrize("call", [
    lambda s, o, i: moe.dispatch(zeros(6, 32), i, 4, zeros(11, 32), stream=s),
    lambda s, o, i: moe.dispatch(zeros(6, 32), i, 4, zeros(12, 32, dtype=F32), stream=s),
    lambda s, o, i: moe.dispatch(zeros(6, 32), zeros(6, 2, dtype=torch.int64), 4, zeros(12, 32), stream=s),
    lambda s, o, i: moe.dispatch(zeros(5, 32), i, 4, zeros(10, 32), stream=s),
    lambda s, o, i: moe.dispatch(zeros(6, 32, dtype=torch.float64), i, 4, zeros(12, 32), stream=s),
    lambda s, o, i: moe.dispatch(zeros(32, 6).t(), i, 4, zeros(12, 32), stream=s),
    lambda s, o, i: moe.dispatch(torch.zeros(6, 32), i, 4, stream=s),
    lambda s, o, i: moe.combine(zeros(12, 32), i, zeros(6, 3, dtype=F32), zeros(6, 32), stream=s),
    lambda s, o, i: moe.combine(zeros(12, 32), i, None, zeros(6, 24), stream=s),
    lambda s, o, i: moe.combine(zeros(12, 32, dtype=torch.float16), i, None, zeros(6, 32), stream=s),
    lambda s, o, i: moe.combine(zeros(12, 32), i, None, out_dtype=torch.float16, stream=s),
    lambda s, o, i: moe.combine_grad(zeros(6, 32), zeros(12, 24), i, None, zeros(12, 32), stream=s),
    lambda s, o, i: moe.combine_grad(zeros(6, 32), zeros(12, 32), i, None, zeros(11, 32), stream=s),
    lambda s, o, i: moe.combine_grad(zeros(5, 32), zeros(12, 32), i, None, zeros(12, 32),
                                                  zeros(5, 2, dtype=F32), stream=s),
    lambda s, o, i: moe.combine_grad(zeros(6, 32), None, i, None, zeros(12, 32), zeros(6, 2, dtype=F32),
                                                  stream=s),
    lambda s, o, i: moe.combine_grad(zeros(6, 32), zeros(12, 32), i, None, zeros(12, 32), num_rows=11,
                                                  stream=s),
    lambda s, o, i: moe.route_topk_grad(i, zeros(6, 2, dtype=F32), zeros(6, 3, dtype=F32), 4,
                                                     zeros(6, 4, dtype=F32), stream=s),
    lambda s, o, i: moe.route_topk_grad(i, zeros(6, 2, dtype=F32), zeros(6, 2, dtype=F32), 4,
                                                     zeros(6, 5, dtype=F32), stream=s),
    lambda s, o, i: moe.quant_int8(zeros(4, 32, dtype=F32), zeros(4, 32, dtype=I8), zeros(4, dtype=F32),
                                               stream=s),
    lambda s, o, i: moe.quant_int8(zeros(4, 32), zeros(4, 16, dtype=I8), zeros(4, dtype=F32), stream=s),
    lambda s, o, i: moe.swiglu_int8(zeros(4, 33), codes=zeros(4, 16, dtype=I8), scales=zeros(4, dtype=F32),
                                                 stream=s),
    lambda s, o, i: moe.grouped_gemm_int8(zeros(7, 32, dtype=I8), zeros(3, 16, 32, dtype=I8),
                                                       zeros(3, 16, dtype=F32), o, zeros(7, 16), stream=s),
    lambda s, o, i: moe.grouped_gemm_int8(zeros(7, 32), zeros(3, 16, 32, dtype=I8),
                                                       zeros(3, 16, dtype=F32), o, zeros(7, 16),
                                                       a_scale=zeros(7, dtype=F32), stream=s),
    lambda s, o, i: moe.grouped_gemm_int8(zeros(7, 32, dtype=I8), zeros(3, 16, 32, dtype=I8),
                                                       zeros(3, 16, dtype=F32), o, zeros(7, 16),
                                                       a_scale=zeros(8, dtype=F32), stream=s),
    lambda s, o, i: moe.grouped_gemm_int8(zeros(7, 32), zeros(3, 16, 32, dtype=torch.uint8),
                                                      zeros(3, 16, dtype=F32), o, zeros(7, 16), stream=s),
    lambda s, o, i: moe.grouped_gemm_int8(zeros(7, 32, dtype=I8), zeros(3, 16, 32, dtype=I8),
                                                       zeros(3, 15, dtype=F32), o, zeros(7, 16),
                                                       a_scale=zeros(7, dtype=F32), stream=s),
])
def test_binding_refuses(calls, monkeypatch, call):  # noqa: F811
    monkeypatch.setattr(moe, "_empty", lambda shape, dtype, *a, **k: zeros(*shape, dtype=dtype))
    with pytest.raises((TypeError, ValueError)):  # a tensor that only says it is on the GPU may be refused as such
        call(Stream(), zeros(4, dtype=I32), zeros(6, 2, dtype=I32))
    assert not calls


@pytest.mark.parametrize("name,call", [
    ("tokens", lambda s, o: moe.dispatch(meta(HUGE, 64), meta(HUGE, 2, dtype=I32), 4, meta(2 * HUGE, 64), stream=s)),
    ("pairs", lambda s, o: moe.dispatch(meta(1 << 30, 64), meta(1 << 30, 4, dtype=I32), 4, meta(1 << 32, 64),
                                        stream=s)),
    ("row bytes", lambda s, o: moe.dispatch(meta(2, 1 << 31), meta(2, 2, dtype=I32), 4, meta(4, 1 << 31), stream=s)),
    ("experts", lambda s, o: moe.dispatch(meta(2, 64), meta(2, 2, dtype=I32), HUGE, meta(4, 64), stream=s)),
    ("first", lambda s, o: moe.dispatch(meta(2, 64), meta(2, 2, dtype=I32), 4, meta(4, 64), first_expert=HUGE,
                                        stream=s)),
    ("rows", lambda s, o: moe.combine(meta(HUGE, 64), meta(2, 2, dtype=I32), None, meta(2, 64), stream=s)),
    ("combined", lambda s, o: moe.combine(meta(2, 64), meta(HUGE, 2, dtype=I32), None, meta(HUGE, 64), stream=s)),
    ("width", lambda s, o: moe.combine(meta(2, HUGE), meta(2, 2, dtype=I32), None, meta(2, HUGE), stream=s)),
    ("grad rows", lambda s, o: moe.combine_grad(meta(2, 64), None, meta(2, 2, dtype=I32), None, meta(HUGE, 64),
                                                num_rows=HUGE, stream=s)),
    ("logits", lambda s, o: moe.route_topk_grad(meta(2, 2, dtype=I32), meta(2, 2, dtype=F32), meta(2, 2, dtype=F32),
                                                HUGE, meta(2, HUGE, dtype=F32), stream=s)),
    ("quantised", lambda s, o: moe.quant_int8(meta(HUGE, 64), meta(HUGE, 64, dtype=I8), meta(HUGE, dtype=F32),
                                              stream=s)),
    ("activated", lambda s, o: moe.swiglu_int8(meta(HUGE, 64), codes=meta(HUGE, 32, dtype=I8),
                                               scales=meta(HUGE, dtype=F32), stream=s)),
    ("product rows", lambda s, o: moe.grouped_gemm_int8(meta(HUGE, 64, dtype=I8), meta(3, 32, 64, dtype=I8),
                                                        meta(3, 32, dtype=F32), o, meta(HUGE, 32),
                                                        a_scale=meta(HUGE, dtype=F32), stream=s)),
    ("divisor", lambda s, o: moe.grouped_gemm_int8(meta(8, 64, dtype=I8), meta(3, 32, 64, dtype=I8),
                                                   meta(3, 32, dtype=F32), o, meta(8, 32), a_scale=meta(8, dtype=F32),
                                                   a_rows=meta(8, dtype=I32), a_div=HUGE, stream=s)),
])
def test_sizes_past_32_bits(calls, name, call):  # noqa: F811
    with pytest.raises(ValueError, match="32 bits"):
        call(Stream(), zeros(4, dtype=I32))
    assert not calls
