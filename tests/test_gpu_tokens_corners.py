"""Corners of the tokens' way to their experts and back: more slots than experts, expert numbers at the end of int32,
the weights' gradient alone, gradients in the rows' place and past 32 bits."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV
from test_gpu_tokens import TYPES, combine_case, layout

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,k,E", [(1, 2, 1), (5, 16, 1), (70, 16, 3), (9, 12, 7), (1000, 5, 4), (33, 16, 15),
                                   (17, 16, 66), (12, 3, 130)])
def test_route_grad_of_equal_ids(M, k, E):
    """Slots that name the same expert, outnumber the experts or name none: their gradients add up."""
    say("route_grad of equal ids M=%d k=%d E=%d" % (M, k, E))
    rng = np.random.default_rng([M, k, E])
    ids = rng.integers(-1, E + 1, (M, k)).astype(np.int32)
    # multiples of 1/16 and whole numbers: w (d - mean) is a multiple of 1/256 below 2^6, exact in fp32 as are its sums
    w = rng.integers(1, 9, (M, k)) / 16.0
    d = rng.integers(-8, 9, (M, k)).astype(np.float64)
    held = (ids >= 0) & (ids < E)
    g = np.where(held, w * (d - (w * d * held).sum(1, keepdims=True)), 0.0)
    want = np.zeros((M, E))
    for t, j in zip(*np.nonzero(held)):
        want[t, ids[t, j]] += g[t, j]
    w[~held], d[~held] = np.nan, np.nan
    got = moe.route_topk_grad(*(torch.from_numpy(v).to(t).to(DEV) for v, t in
                                ((ids, torch.int32), (w, torch.float32), (d, torch.float32))), E)
    assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("M", [40, 3000, 40000])  # the three ways of counting pairs
@pytest.mark.parametrize("E,back", [(8, 4), (512, 1), (512, 511), (300, 300)])
def test_dispatch_at_the_end_of_int32(M, E, back):
    """No id is an expert's of a range that would go on behind 2^31, the lowest int32s among them."""
    say("dispatch M=%d of E=%d experts from 2^31 - %d" % (M, E, back))
    rng = np.random.default_rng([M, E, back])
    first, lowest, highest = 2 ** 31 - back, -2 ** 31, 2 ** 31 - 1
    near = [highest - rng.integers(0, 600, (M, 2)), lowest + rng.integers(0, 600, (M, 2)),
            np.tile([highest, lowest], (M, 1)), rng.integers(-2, 600, (M, 2))]
    ids = np.choose(rng.integers(0, 4, (M, 2)), near).astype(np.int32)
    got = moe.dispatch(None, torch.from_numpy(ids).to(DEV), E, first_expert=first)[1:]
    for t, want in zip(got, layout(ids, E, first)):
        assert np.array_equal(t.cpu().numpy(), want)


@pytest.mark.parametrize("M,k,E,H", [(1, 1, 1, 8), (600, 8, 8, 64), (50, 3, 8, 128), (33, 16, 16, 256), (77, 3, 7, 520),
                                     (130, 6, 64, 1024), (130, 6, 64, 1032), (9, 2, 4, 14336), (20001, 2, 9, 1040)])
@pytest.mark.parametrize("dy_type,rows_type", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("weighted", [True, False])
def test_gradient_of_the_weights_alone(M, k, E, H, dy_type, rows_type, weighted):
    """What a router that is trained alone takes: the bits of the call that makes both gradients."""
    say("dweights alone %s" % ((M, k, E, H, dy_type, rows_type, weighted),))
    rng, rows, pos, valid, w = combine_case(M, k, E, H, rows_type, "bf16", weighted, 0.3, 2)
    dy = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(TYPES[dy_type]).to(DEV)
    rows, pos = rows.to(DEV), torch.from_numpy(pos).to(DEV)
    w = None if w is None else torch.from_numpy(w).to(DEV)
    _, want = moe.combine_grad(dy, rows, pos, w)
    canvas = torch.full((M, k), 7.0, device=DEV)
    none, dw = moe.combine_grad(dy, rows, pos, w, dweights=canvas, out_dtype=None)
    assert none is None and dw.data_ptr() == canvas.data_ptr() and torch.equal(dw, want)
    none, made = moe.combine_grad(dy, rows, pos, w, out_dtype=None)
    assert none is None and torch.equal(made, want)


def test_given_rows_take_the_gradient_whatever_out_dtype_is():
    dy = torch.ones(3, 64, device=DEV)
    pos = torch.arange(6, dtype=torch.int32, device=DEV).view(3, 2)
    drows, _ = moe.combine_grad(dy, None, pos, None, torch.zeros(6, 64, device=DEV), out_dtype=None)
    assert bool((drows == 1).all())


@pytest.mark.parametrize("M,k,E,H", [(600, 8, 8, 64), (33, 16, 16, 256), (77, 3, 7, 520), (130, 6, 64, 1032),
                                     (9, 2, 4, 14336), (20001, 2, 9, 1040)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_gradient_in_the_rows_place(M, k, E, H, kind):
    say("drows in place of rows %s" % ((M, k, E, H, kind),))
    rng, rows, pos, valid, w = combine_case(M, k, E, H, kind, kind, True, 0.3, 3)
    dy = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(TYPES[kind]).to(DEV)
    pos, w = torch.from_numpy(pos).to(DEV), torch.from_numpy(w).to(DEV)
    wide = torch.full((M * k, H + 16), 7.0, dtype=TYPES[kind], device=DEV)
    place = wide[:, 8:H + 8]
    place.copy_(rows)
    apart = place.clone()
    want, want_dw = moe.combine_grad(dy, place, pos, w, apart)
    drows, dw = moe.combine_grad(dy, place, pos, w, place)
    assert drows.data_ptr() == place.data_ptr()
    as_bytes = [t.contiguous().view(torch.uint8) for t in (place, want)]  # rows without a place hold NaN
    assert torch.equal(*as_bytes) and torch.equal(dw, want_dw)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, H + 8:] == 7).all())


@pytest.mark.parametrize("alone", [False, True])
def test_weights_gradient_past_32_bits(alone):
    """Rows of 5 GB and their gradient of 5 GB beside them: places past 2^31 and 2^32 bytes, in both."""
    M, k, E, H = 40000, 8, 32, 8192
    g = torch.Generator(device=DEV).manual_seed(6)
    # whole numbers, each row's sum of products below 2^24: exact in fp32 in any order
    dy = torch.randint(-4, 5, (M, H), generator=g, device=DEV, dtype=torch.int32).to(torch.bfloat16)
    ids = torch.topk(torch.rand(M, E, generator=g, device=DEV), k, 1).indices.to(torch.int32)
    rows, off, pos, pairs = moe.dispatch(dy, ids, E)
    # each row times a factor of its own place, so that another row's would show
    factor = (torch.arange(M * k, device=DEV) % 13 - 6).to(torch.bfloat16)
    rows *= factor[:, None]
    w = torch.rand(M, k, generator=g, device=DEV)
    drows, dw = moe.combine_grad(dy, rows, pos, w, out_dtype=None if alone else torch.bfloat16)
    square = dy.float().square().sum(1, keepdim=True)
    assert float(square.max()) * 6 < 2 ** 24
    assert torch.equal(dw, square * factor.float()[pos.long()])
    if alone:
        assert drows is None
        return
    for i in range(0, M * k, 40000):
        f = pairs[i:i + 40000].long()
        assert torch.equal(drows[i:i + 40000], (w.view(-1)[f, None] * dy[f // k].float()).to(torch.bfloat16))
