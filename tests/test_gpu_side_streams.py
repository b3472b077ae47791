"""Memory of the calls that are given another stream than the current one: what
a call allocates for that stream must not be memory that work queued on the
current stream still uses."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV, bf16, offsets_of

pytestmark = pytest.mark.gpu

R, E, N, K = 512, 4, 512, 256


@pytest.fixture(scope="module")
def ops():
    rng = np.random.default_rng(1)
    off = torch.from_numpy(offsets_of([100, 200, 0, 212])).to(DEV)
    a, dy = bf16(rng, R, K).to(DEV), bf16(rng, R, N).to(DEV)
    w = bf16(rng, E, N, K, scale=K ** -0.5).to(DEV)
    w4 = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)).to(DEV)
    s4 = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device=DEV)
    _, codes, scales = moe.swiglu_checkpoint(dy)
    dh = dy[:, :N // 2].contiguous()
    calls = {
        "product": lambda s: moe.grouped_gemm(a, w, off, stream=s),
        "input gradient": lambda s: moe.grouped_gemm_dgrad(dy, w, off, stream=s),
        "weight gradient": lambda s: moe.grouped_gemm_wgrad(dy, a, off, stream=s),
        "4-bit product": lambda s: moe.grouped_gemm_w4(a, w4, s4, off, stream=s),
        "checkpoint": lambda s: moe.swiglu_checkpoint(dy, stream=s),
        "checkpoint gradient": lambda s: moe.swiglu_checkpoint_grad(codes, scales, dh, stream=s),
    }
    torch.cuda.synchronize()
    return calls


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


def stream_forms(s):
    """The ways a caller names a stream."""
    return {"torch stream": s, "handle": s.cuda_stream, "external": torch.cuda.ExternalStream(s.cuda_stream)}


CALLS = ["product", "input gradient", "weight gradient", "4-bit product", "checkpoint", "checkpoint gradient"]


@pytest.mark.parametrize("form", ["torch stream", "handle", "external"])
@pytest.mark.parametrize("name", CALLS)
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


def test_a_dropped_output_is_not_handed_out_while_the_current_stream_reads_it(ops):
    side = torch.cuda.Stream()
    big = torch.zeros(64 << 20, device=DEV)
    want = ops["product"](None).float().sum()
    torch.cuda.synchronize()
    y = ops["product"](side)
    side.synchronize()
    for _ in range(40):
        big.add_(1.0)
    got = y.float().sum()
    del y
    with torch.cuda.stream(side):
        junk = [torch.full((R, N), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


def test_default_stream_by_its_handle(ops):
    # handle 0 is the default stream also while another one is current
    want = ops["product"](None)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = ops["product"](torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_side_stream_call_inside_a_capture(ops):
    # the call's stream is forked from the capturing one and joined again; the graph's outputs are its own memory
    want = ops["product"](None)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        y = ops["product"](side)
        cur.wait_stream(side)
        z = y + 0
    for _ in range(4):
        y.zero_()
        z.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want)
        ops["checkpoint"](None)  # eager work between the replays
        torch.cuda.synchronize()


def layer_calls():
    M, LE, k, H, I = 300, 16, 4, 512, 256
    rng = np.random.default_rng(2)
    x, logits = bf16(rng, M, H).to(DEV), torch.from_numpy(rng.standard_normal((M, LE)).astype(np.float32)).to(DEV)
    w13 = bf16(rng, LE, 2 * I, H, scale=H ** -0.5).to(DEV)
    w2, rw = bf16(rng, LE, H, I, scale=I ** -0.5).to(DEV), bf16(rng, LE, H).to(DEV)
    ids, _ = moe.route_topk(logits, k)
    data, scale = logits.flatten().contiguous(), torch.ones(1, device=DEV)

    def align(s):
        al = moe.align(ids, LE, 16, stream=s)
        return [al["counts"], al["offsets"], al["num_padded"]]

    return {
        "route_topk": lambda s: moe.route_topk(logits, k, stream=s),
        "router_logits": lambda s: moe.router_logits(x, rw, stream=s),
        "align": align,
        "quant_e4m3": lambda s: moe.quant_e4m3(data, scale, stream=s),
        "fused_forward": lambda s: moe.fused_forward(x, logits, w13, w2, k, "bf16", stream=s),
    }


@pytest.mark.parametrize("name", ["route_topk", "router_logits", "align", "quant_e4m3", "fused_forward"])
def test_the_layers_own_calls(name):
    # the same of the layer's calls; the workspace that fused_forward makes would be among what overwrites `tmp`
    say("side-stream memory: %s" % name)
    call = layer_calls()[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    side, big = torch.cuda.Stream(), torch.zeros(64 << 20, device=DEV)
    sizes = [t.numel() * t.element_size() for t in want] + [
        moe.workspace_size(300, 16, 512, 256, 4, "bf16")] * (name == "fused_forward")
    tmp = [torch.full((n,), 3 + i, dtype=torch.uint8, device=DEV) for i, n in enumerate(sizes)]
    torch.cuda.synchronize()
    for _ in range(40):
        big.add_(1.0)
    sums = [t.to(torch.int32).sum() for t in tmp]
    freed = [t.data_ptr() for t in tmp]
    del tmp
    got = tensors(call(side))
    for g in got:
        b = g.numel() * g.element_size()
        assert not any(p < g.data_ptr() + b and g.data_ptr() < p + n for p, n in zip(freed, sizes)), \
            "an output lies in memory that queued work reads"
    torch.cuda.synchronize()
    assert [int(s) for s in sums] == [(3 + i) * n for i, n in enumerate(sizes)]
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
