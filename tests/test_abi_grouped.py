"""Host-only checks of the grouped products' and the checkpointed activation's
entry points (no GPU needed): every refusal the header documents comes back
before anything is enqueued."""
import ctypes
import os

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 1 << 20  # a pointer that is never followed


@pytest.fixture(scope="module")
def m():
    import moe_layer_align_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.fail("libmoe_mi355x.so is not built; run __graft_entry__.build()")
    m.load()
    return m


def rows(m, width, n=10, **kw):
    d = dict(data=P, stride=width, rows=n, div=1, ids=None)
    d.update(kw)
    return m._Rows(**d)


def gemm(m, fn="moe_grouped_gemm", in_=None, out=None, null=False, **kw):
    d = dict(R=10, E=4, N=64, K=128, offsets=P, weight=0, w=P, w_scale=None, out_type=0)
    d.update(kw)
    src, dst = (d["N"], d["K"]) if fn.endswith("dgrad") else (d["K"], d["N"])
    a = m._GroupedArgs(in_=rows(m, src, **(in_ or {})), out=rows(m, dst, **(out or {})), **d)
    return getattr(m.load(), fn)(None if null else ctypes.byref(a), None)


BAD = [
    (dict(R=-1), INVALID), (dict(E=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID),
    (dict(offsets=None), INVALID), (dict(offsets=P + 2), INVALID), (dict(w=None), INVALID), (dict(w=P + 8), INVALID),
    (dict(w_scale=P), INVALID), (dict(weight=3), INVALID), (dict(weight=-1), INVALID), (dict(out_type=2), INVALID),
    (dict(E=513), UNSUPPORTED), (dict(R=1 << 26, in_=dict(n=1 << 26), out=dict(n=1 << 26)), UNSUPPORTED), (dict(N=12), UNSUPPORTED), (dict(K=132), UNSUPPORTED),
    (dict(N=1 << 16, K=1 << 14), UNSUPPORTED),
    (dict(in_=dict(data=None)), INVALID), (dict(in_=dict(data=P + 8)), INVALID), (dict(in_=dict(stride=64 - 8)), INVALID),
    (dict(in_=dict(stride=132)), INVALID), (dict(in_=dict(stride=1 << 20)), UNSUPPORTED),
    (dict(in_=dict(n=9)), INVALID), (dict(in_=dict(div=2)), INVALID), (dict(in_=dict(ids=P, div=0)), INVALID),
    (dict(in_=dict(ids=P + 1)), INVALID), (dict(in_=dict(n=-1, ids=P)), INVALID),
    (dict(in_=dict(ids=P, n=1 << 24, stride=128)), UNSUPPORTED),
    (dict(out=dict(data=None)), INVALID), (dict(out=dict(data=P + 4)), INVALID), (dict(out=dict(n=9)), INVALID),
    (dict(out=dict(ids=P, div=2)), INVALID), (dict(out=dict(stride=56)), INVALID), (dict(out=dict(stride=140)), INVALID),
]


@pytest.mark.parametrize("fn", ["moe_grouped_gemm", "moe_grouped_gemm_dgrad"])
@pytest.mark.parametrize("kw,code", BAD)
def test_gemm_refusals(m, fn, kw, code):
    assert gemm(m, fn, **kw) == code


def test_gemm_w4_refusals(m):
    assert gemm(m, weight=1) == INVALID                        # no scales
    assert gemm(m, weight=2, w_scale=P + 1) == INVALID          # bf16 scales at an odd address
    assert gemm(m, weight=1, w_scale=P, K=136) == UNSUPPORTED   # half a group
    assert gemm(m, weight=2, w_scale=P, K=96) == UNSUPPORTED
    assert gemm(m, "moe_grouped_gemm_dgrad", weight=1, w_scale=P) == UNSUPPORTED


def test_nothing_to_do(m):
    assert gemm(m, R=0, offsets=None, w=None) == OK
    assert gemm(m, null=True) == INVALID
    lib = m.load()
    assert lib.moe_swiglu_checkpoint(None, 0, None, 0, 64, None, None, None, None, None) == OK
    assert lib.moe_swiglu_checkpoint_grad(None, None, None, None, 0, 64, None, None, None, None, None) == OK


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INVALID), (dict(N=0), INVALID), (dict(E=600), UNSUPPORTED), (dict(N=20), UNSUPPORTED),
    (dict(offsets=None), INVALID), (dict(dw=None), INVALID), (dict(dw=P + 4), INVALID), (dict(out_type=7), INVALID),
    (dict(accumulate=2), INVALID), (dict(accumulate=1, out_type=0), INVALID), (dict(dy=dict(data=None)), INVALID),
    (dict(dy=dict(n=9)), INVALID), (dict(in_=dict(n=9)), INVALID), (dict(in_=dict(ids=P, div=-1)), INVALID),
    (dict(dy=dict(stride=1 << 20)), UNSUPPORTED), (dict(in_=dict(ids=P, n=1 << 24)), UNSUPPORTED),
])
def test_wgrad_refusals(m, kw, code):
    kw = dict(kw)
    dy, in_ = kw.pop("dy", {}), kw.pop("in_", {})
    d = dict(R=10, E=4, N=64, K=128, offsets=P, dw=P, out_type=1, accumulate=0)
    d.update(kw)
    a = m._GroupedWgradArgs(dy=rows(m, d["N"], **dy), in_=rows(m, d["K"], **in_), **d)
    assert m.load().moe_grouped_gemm_wgrad(ctypes.byref(a), None) == code
    assert m.load().moe_grouped_gemm_wgrad(None, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INVALID), (dict(I=0), INVALID), (dict(I=12), UNSUPPORTED), (dict(I=1 << 19), UNSUPPORTED),
    (dict(R=1 << 30, I=4096), UNSUPPORTED), (dict(gu=None), INVALID), (dict(gu=P + 2), INVALID),
    (dict(stride=120), INVALID), (dict(stride=132), INVALID), (dict(stride=1 << 20), UNSUPPORTED),
    (dict(h=None, codes=None, scales=None), INVALID), (dict(scales=None), INVALID), (dict(codes=None), INVALID),
    (dict(codes=P + 8), INVALID), (dict(h=P + 8), INVALID), (dict(weight=P + 2), INVALID), (dict(num=P + 1), INVALID),
])
def test_checkpoint_refusals(m, kw, code):
    d = dict(gu=P, stride=128, weight=None, R=4, I=64, num=None, h=P, codes=P, scales=P)
    d.update(kw)
    assert m.load().moe_swiglu_checkpoint(d["gu"], d["stride"], d["weight"], d["R"], d["I"], d["num"], d["h"],
                                          d["codes"], d["scales"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), INVALID), (dict(I=-8), INVALID), (dict(I=20), UNSUPPORTED), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(dh=None), INVALID), (dict(dgu=None), INVALID), (dict(dgu=P + 8), INVALID),
    (dict(h=P + 4), INVALID), (dict(dweight=P + 2), INVALID), (dict(R=1 << 30, I=4096), UNSUPPORTED),
])
def test_checkpoint_grad_refusals(m, kw, code):
    d = dict(codes=P, scales=P, dh=P, weight=None, R=4, I=64, num=None, dgu=P, h=P, dweight=P)
    d.update(kw)
    assert m.load().moe_swiglu_checkpoint_grad(d["codes"], d["scales"], d["dh"], d["weight"], d["R"], d["I"], d["num"],
                                               d["dgu"], d["h"], d["dweight"], None) == code


def test_binding_refuses_cpu_tensors(m):
    a, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(1, 32, 64, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.grouped_gemm(a, w, off)
    with pytest.raises(ValueError):
        m.grouped_gemm_wgrad(a, a, off)
    with pytest.raises(ValueError):
        m.swiglu_checkpoint(a)


@pytest.mark.parametrize("R,I", [(1 << 26, 8), (1 << 25, 1032), (1 << 24, 2048), ((1 << 31) - 1, 8)])
def test_activation_sizes(m, R, I):
    # more rows or elements than a grid of 2^32 threads covers
    assert m.load().moe_swiglu_checkpoint(P, 2 * I, None, R, I, None, P, P, P, None) == UNSUPPORTED
    assert m.load().moe_swiglu_checkpoint_grad(P, P, P, None, R, I, None, P, P, P, None) == UNSUPPORTED
