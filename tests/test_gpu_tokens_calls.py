"""How dispatch, combine, their gradients and the products in 8-bit integers are
called: on side streams, several at once, captured into graphs and replayed, on
views, with equal positions, on buffers past 32-bit offsets, on random sizes."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV, bf16
from test_gpu_grouped_calls import same
from test_gpu_side_streams import stream_forms, tensors
from test_gpu_tokens import layout, routing

pytestmark = pytest.mark.gpu


class Layer:
    """One pass of a layer in 8-bit integers, the gradients of its combine and its router, and a bf16 product on the
    copied rows; what it makes is kept under names."""

    def __init__(self, seed, M, E, k, H=128, I=80):
        rng = np.random.default_rng(seed)
        self.E, self.k, self.H, self.I = E, k, H, I
        self.x, self.dy = bf16(rng, M, H).to(DEV), bf16(rng, M, H).to(DEV)
        self.logits = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32)).to(DEV)
        self.w13, self.s13 = moe.quant_int8(bf16(rng, E * 2 * I, H, scale=H ** -0.5).to(DEV))
        self.w2, self.s2 = moe.quant_int8(bf16(rng, E * H, I, scale=I ** -0.5).to(DEV))
        self.wb = bf16(rng, E, 64, H).to(DEV)

    def run(self, stream=None):
        E, H, I, kw = self.E, self.H, self.I, dict(stream=stream)
        o = {}
        o["ids"], o["w"] = moe.route_topk(self.logits, self.k, **kw)
        o["rows"], o["off"], o["pos"], o["pairs"] = moe.dispatch(self.x, o["ids"], E, **kw)
        o["codes"], o["scales"] = moe.quant_int8(o["rows"], **kw)
        w13, s13 = self.w13.view(E, 2 * I, H), self.s13.view(E, 2 * I)
        w2, s2 = self.w2.view(E, H, I), self.s2.view(E, H)
        o["gu"] = moe.grouped_gemm_int8(o["codes"], w13, s13, o["off"], a_scale=o["scales"], **kw)
        o["gu2"] = moe.grouped_gemm_int8(self.x, w13, s13, o["off"], a_rows=o["pairs"], a_div=self.k, **kw)
        o["h"], o["hs"] = moe.swiglu_int8(o["gu"], num_rows=o["off"][E:], **kw)
        o["d"] = moe.grouped_gemm_int8(o["h"], w2, s2, o["off"], a_scale=o["hs"], **kw)
        o["b"] = moe.grouped_gemm(o["rows"], self.wb, o["off"], **kw)
        o["y"] = moe.combine(o["d"], o["pos"], o["w"], **kw)
        o["drows"], o["dw"] = moe.combine_grad(self.dy, o["d"], o["pos"], o["w"], **kw)
        o["dlogits"] = moe.route_topk_grad(o["ids"], o["w"], o["dw"], E, **kw)
        o["dx"] = moe.combine(o["drows"], o["pos"], **kw)
        return o


# the three ways of counting pairs, products of few and of many rows
LAYERS = [dict(M=40, E=8, k=2), dict(M=3000, E=6, k=2), dict(M=4096, E=130, k=8), dict(M=9000, E=16, k=1, H=64, I=48)]


def clones(o):
    return {n: t.clone() for n, t in o.items()}


def test_same_bits_on_side_streams_and_at_once():
    layers = [Layer(i, **kw) for i, kw in enumerate(LAYERS)]
    alone = []
    for s in layers:
        first = clones(s.run())
        torch.cuda.synchronize()
        same(first, s.run(), "a second time")
        alone.append(first)
    for s in alone:
        same({"gu": s["gu"]}, {"gu": s["gu2"]}, "codes made in the call")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for rep in range(3):
        say("layers at once, round %d" % rep)
        got = [s.run(st) for s, st in zip(layers, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            same(a, b, "side stream")


@pytest.mark.parametrize("kw", LAYERS, ids=str)
def test_captured_and_replayed(kw):
    s = Layer(4, **kw)
    want = clones(s.run())
    other = Layer(5, **kw)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = s.run()
    with torch.cuda.graph(g2):
        got2 = other.run()
    for rep in range(4):
        say("replay %d of %s" % (rep, kw))
        for t in list(got.values()) + list(got2.values()):
            t.zero_()
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        same(want, got, "replay %d" % rep)
        same(other.run(), got2, "the other graph's replay %d" % rep)  # eager work of the same kernels in between
        torch.cuda.synchronize()
    # new inputs, and another routing, in the same buffers
    s.x.copy_(other.x)
    s.logits.copy_(other.logits)
    g.replay()
    torch.cuda.synchronize()
    got = clones(got)
    same(s.run(), got, "replay on new inputs")


@pytest.fixture(scope="module")
def ops():
    s = Layer(9, M=900, E=20, k=8)
    o = s.run()
    E, H, I = s.E, s.H, s.I
    w13, s13 = s.w13.view(E, 2 * I, H), s.s13.view(E, 2 * I)
    torch.cuda.synchronize()
    return {
        "dispatch": lambda st: moe.dispatch(s.x, o["ids"], E, stream=st),
        "combine": lambda st: moe.combine(o["d"], o["pos"], o["w"], stream=st),
        "combine_grad": lambda st: moe.combine_grad(s.dy, o["d"], o["pos"], o["w"], stream=st),
        "route_grad": lambda st: moe.route_topk_grad(o["ids"], o["w"], o["dw"], E, stream=st),
        "quant": lambda st: moe.quant_int8(s.x, stream=st),
        "swiglu": lambda st: moe.swiglu_int8(o["gu"], stream=st),
        "product": lambda st: moe.grouped_gemm_int8(o["codes"], w13, s13, o["off"], a_scale=o["scales"], stream=st),
        "bf16 rows": lambda st: moe.grouped_gemm_int8(s.x, w13, s13, o["off"], a_rows=o["pairs"], a_div=s.k, stream=st),
    }


@pytest.mark.parametrize("form", ["torch stream", "handle", "external"])
@pytest.mark.parametrize("name", ["dispatch", "combine", "combine_grad", "route_grad", "quant", "swiglu", "product",
                                  "bf16 rows"])
def test_outputs_do_not_take_memory_that_the_current_stream_may_use(ops, name, form):
    say("side-stream memory: %s, %s" % (name, form))
    want = [t.clone() for t in tensors(ops[name](None))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.zeros(64 << 20, device=DEV)
    tmp = [torch.full_like(t.view(torch.uint8), 3 + i) for i, t in enumerate(want)]
    torch.cuda.synchronize()
    # the current stream: long work, then reads of the buffers, which are freed at once
    for _ in range(40):
        big.add_(1.0)
    sums = [t.view(torch.uint8).to(torch.int32).sum() for t in tmp]
    freed, sizes = [t.data_ptr() for t in tmp], [t.numel() for t in tmp]
    expect = [(3 + i) * n for i, n in enumerate(sizes)]
    del tmp
    got = tensors(ops[name](stream_forms(side)[form]))
    for g in got:
        b = g.numel() * g.element_size()
        assert not any(p < g.data_ptr() + b and g.data_ptr() < p + n for p, n in zip(freed, sizes)), \
            "an output lies in memory that queued work reads"
    torch.cuda.synchronize()
    assert [int(s) for s in sums] == expect
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


def test_views_and_odd_addresses():
    rng = np.random.default_rng(3)
    x = bf16(rng, 50, 96).to(DEV)
    ids = torch.from_numpy(routing(rng, 50, 2, 5)).to(DEV)
    rows, off, pos, pairs = moe.dispatch(x, ids, 5)
    w = torch.rand(51, 2, device=DEV)[1:]
    # every second row, columns from 16 bytes on
    wide = torch.zeros(100, 104, dtype=torch.bfloat16, device=DEV)
    view = wide[::2, 8:]
    view.copy_(x)
    assert torch.equal(moe.dispatch(view, ids, 5)[0], rows)
    assert torch.equal(moe.quant_int8(view)[0], moe.quant_int8(x)[0])
    y = moe.combine(rows, pos, w)
    big = torch.zeros(100, 104, dtype=torch.bfloat16, device=DEV)
    big[:, 8:].copy_(rows)
    assert torch.equal(moe.combine(big[:, 8:], pos, w), y)
    assert torch.equal(moe.combine_grad(view, big[:, 8:], pos, w)[1], moe.combine_grad(x, rows, pos, w)[1])
    off_by_two = wide.view(-1)[1:1 + 50 * 96].view(50, 96)
    for call in (lambda: moe.dispatch(off_by_two, ids, 5),
                 lambda: moe.combine(off_by_two, pos[:25], w[:25].contiguous()),
                 lambda: moe.combine_grad(off_by_two, rows, pos, w.contiguous()), lambda: moe.quant_int8(off_by_two),
                 lambda: moe.dispatch(x[:, :90], ids, 5), lambda: moe.quant_int8(x[:, :88])):
        with pytest.raises(moe.MoEError):
            call()
    with pytest.raises(ValueError):
        moe.combine(rows, pos, torch.rand(50, 4, device=DEV)[:, ::2])


def test_equal_positions():
    """A row that several slots name counts in each; its gradient is one of theirs."""
    rng = np.random.default_rng(5)
    rows = bf16(rng, 3, 64).to(DEV)
    pos = torch.tensor([[0, 0], [2, 0]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, 0.25], [2.0, 1.0]], device=DEV)
    y = moe.combine(rows, pos, w, out_dtype=torch.float32)
    r = rows.float()
    assert torch.equal(y, torch.stack((0.75 * r[0], 2.0 * r[2] + r[0])))
    dy = bf16(rng, 2, 64).to(DEV)
    drows, dw = moe.combine_grad(dy, rows, pos, w)
    one_of = [(w[t, j] * dy[t].float()).to(torch.bfloat16) for t, j in ((0, 0), (0, 1), (1, 1))]
    assert any(torch.equal(drows[0], v) for v in one_of)
    assert torch.equal(drows[2], (2.0 * dy[1].float()).to(torch.bfloat16))
    assert dw[0, 0] == dw[0, 1]


def test_buffers_past_32_bits():
    """Rows of 5 GB: places past 2^31 and 2^32 bytes."""
    M, k, E, H = 40000, 8, 32, 8192
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randint(-99, 99, (M, H), generator=g, device=DEV, dtype=torch.int32).to(torch.bfloat16)
    ids = torch.topk(torch.rand(M, E, generator=g, device=DEV), k, 1).indices.to(torch.int32)
    rows, off, pos, pairs = moe.dispatch(x, ids, E)
    r_off, r_pos, r_pairs = layout(ids.cpu().numpy(), E)
    assert np.array_equal(pos.cpu().numpy(), r_pos) and np.array_equal(pairs.cpu().numpy(), r_pairs)
    assert off.tolist() == r_off.tolist()
    for i in range(0, M * k, 40000):
        assert torch.equal(rows[i:i + 40000], x[pairs[i:i + 40000].long() // k])
    # whole numbers times powers of two: exact
    w = torch.full((M, k), 0.125, device=DEV)
    assert torch.equal(moe.combine(rows, pos, w), x)
    drows, dw = moe.combine_grad(x, rows, pos, w, rows)
    for i in range(0, M * k, 40000):
        assert torch.equal(drows[i:i + 40000], 0.125 * x[pairs[i:i + 40000].long() // k])


@pytest.mark.parametrize("R,E,N,K,dtype", [(70000, 2, 16384, 16, torch.float32), (40, 9, 65536, 8176, torch.bfloat16)])
def test_products_past_32_bits(R, E, N, K, dtype):
    """Results of 4.6 GB; weights of 4.8 GB."""
    g = torch.Generator(device=DEV).manual_seed(2)
    a = torch.randint(-9, 9, (R, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-9, 9, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    bounds = [R * e // E for e in range(E + 1)]
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    one = torch.ones(E, N, device=DEV)
    y = moe.grouped_gemm_int8(a, w, one, off, a_scale=torch.full((R,), 0.5, device=DEV), out_dtype=dtype)
    for e in range(E):
        for i in range(bounds[e], bounds[e + 1], 8192):
            s = slice(i, min(i + 8192, bounds[e + 1]))
            # sums of at most 2^23: exact in fp32
            assert torch.equal(y[s], (0.5 * (a[s].float() @ w[e].float().t())).to(dtype))


@pytest.mark.parametrize("seed", range(24))
def test_random_sizes(seed):
    """Sizes over the range, chosen by the seed; whole numbers, so that every result but the rounded ones is exact."""
    rng = np.random.default_rng([77, seed])
    k = int(rng.integers(1, 17))
    E = int(np.exp(rng.uniform(np.log(k), np.log(512))))
    E = max(E, k)
    M = max(1, int(np.exp(rng.uniform(0, np.log(20000 // k)))))
    H = 16 * max(1, int(np.exp(rng.uniform(0, np.log(200)))))
    first = int(rng.integers(0, 3))
    say("random sizes %d: M=%d k=%d E=%d H=%d first=%d" % (seed, M, k, E, H, first))
    ids = routing(rng, M, k, E, first, float(rng.choice([0.0, 0.1])), float(rng.choice([0.0, 1.0])), seed % 3 == 0)
    x = torch.from_numpy(rng.integers(-8, 9, (M, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    rows, off, pos, pairs = moe.dispatch(x, torch.from_numpy(ids).to(DEV), E, first_expert=first)
    r_off, r_pos, r_pairs = layout(ids, E, first)
    assert np.array_equal(off.cpu().numpy(), r_off) and np.array_equal(pos.cpu().numpy(), r_pos)
    assert np.array_equal(pairs.cpu().numpy(), r_pairs)
    n = int(r_off[-1])
    assert torch.equal(rows[:n], x[torch.from_numpy(r_pairs[:n] // k).to(DEV)])
    w = torch.from_numpy(rng.integers(-4, 5, (M, k)).astype(np.float32)).to(DEV)
    valid = pos >= 0
    wv = torch.where(valid, w, 0.0)
    y = moe.combine(rows, pos, w, out_dtype=torch.float32)
    assert torch.equal(y, wv.sum(1, keepdim=True) * x.float())  # every row is the token's own
    dy = torch.from_numpy(rng.integers(-4, 5, (M, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    drows, dw = moe.combine_grad(dy, rows, pos, w)
    assert torch.equal(dw, torch.where(valid, (dy.float() * x.float()).sum(1, keepdim=True), 0.0))
    token = torch.from_numpy(r_pairs[:n] // k).to(DEV)
    flat = torch.from_numpy(r_pairs[:n]).to(DEV)
    assert torch.equal(drows[:n].float(), w.view(-1)[flat, None] * dy[token].float())
    # a product with the codes of the rows, small enough to be exact
    N = 8 * int(rng.integers(1, 40))
    wt = torch.from_numpy(rng.integers(-3, 4, (E, N, H), dtype=np.int8)).to(DEV)
    codes = x.to(torch.int8)
    pid = torch.where(pairs >= 0, pairs, M * k)
    z = moe.grouped_gemm_int8(codes, wt, torch.ones(E, N, device=DEV), off, a_scale=torch.ones(M, device=DEV),
                              a_rows=pid, a_div=k, out_dtype=torch.float32)
    for e in range(E):
        s = slice(int(r_off[e]), int(r_off[e + 1]))
        if s.start < s.stop:
            assert torch.equal(z[s], rows[s].float() @ wt[e].float().t())
