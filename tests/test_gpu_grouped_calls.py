"""How the grouped products and the checkpointed activation are called: on side
streams, several at once, captured into a graph and replayed, with outputs that
are used again, at the corners of their arguments' rules."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV, bf16, check, f64, offsets_of, w4_values

pytestmark = pytest.mark.gpu


class Step:
    """One training step of a layer's expert half and a 4-bit product on fixed
    buffers; run() enqueues it, reads nothing back and allocates nothing."""

    def __init__(self, seed, M=90, E=6, k=2, H=264, I=136, block=16):
        rng = np.random.default_rng(seed)
        self.k, self.E = k, E
        self.x, self.dy = bf16(rng, M, H).to(DEV), bf16(rng, M, H).to(DEV)
        self.w13 = bf16(rng, E, 2 * I, H, scale=H ** -0.5).to(DEV)
        self.w2 = bf16(rng, E, H, I, scale=I ** -0.5).to(DEV)
        logits = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32)).to(DEV)
        ids, _ = moe.route_topk(logits, k)
        al = moe.align(ids, E, block)
        self.off, self.rows = al["offsets"], al["sorted_ids"]
        R = self.rows.numel()
        self.num = self.off[E:]
        self.wt = torch.from_numpy(rng.uniform(0.1, 1, R).astype(np.float32)).to(DEV)
        kw = dict(device=DEV, dtype=torch.bfloat16)
        self.gu, self.h = torch.zeros(R, 2 * I, **kw), torch.zeros(R, I, **kw)
        self.codes = torch.zeros(R, 2 * I, dtype=torch.uint8, device=DEV)
        self.scales = torch.zeros(R, 2, -(-I // 32), dtype=torch.uint8, device=DEV)
        self.o, self.dxp = torch.zeros(M * k, H, **kw), torch.zeros(M * k, H, **kw)
        self.dh, self.dgu, self.hw = torch.zeros(R, I, **kw), torch.zeros(R, 2 * I, **kw), torch.zeros(R, I, **kw)
        self.dwt = torch.zeros(R, device=DEV)
        self.dw13 = torch.zeros(E, 2 * I, H, device=DEV)
        self.dw2 = torch.zeros(E, H, I, device=DEV)
        self.K4 = H // 32 * 32
        self.w4 = torch.from_numpy(rng.integers(0, 256, (E, 2 * I, self.K4 // 2), dtype=np.uint8)).to(DEV)
        self.s4 = torch.from_numpy(rng.integers(115, 130, (E, 2 * I, self.K4 // 32), dtype=np.uint8)).to(DEV)
        self.y4 = torch.zeros(R, 2 * I, **kw)

    OUT = ("gu", "h", "codes", "scales", "o", "dh", "dgu", "hw", "dwt", "dw13", "dw2", "dxp", "y4")

    def run(self, stream=None):
        kw = dict(stream=stream)
        moe.grouped_gemm(self.x, self.w13, self.off, self.gu, a_rows=self.rows, a_div=self.k, **kw)
        moe.swiglu_checkpoint(self.gu, self.wt, num_rows=self.num, h=self.h, codes=self.codes, scales=self.scales, **kw)
        moe.grouped_gemm(self.h, self.w2, self.off, self.o, out_rows=self.rows, **kw)
        moe.grouped_gemm_dgrad(self.dy, self.w2, self.off, self.dh, dy_rows=self.rows, dy_div=self.k, **kw)
        moe.swiglu_checkpoint_grad(self.codes, self.scales, self.dh, self.wt, num_rows=self.num, dgu=self.dgu, h=self.hw,
                                   dweight=self.dwt, **kw)
        moe.grouped_gemm_wgrad(self.dy, self.hw, self.off, self.dw2, dy_rows=self.rows, dy_div=self.k, **kw)
        moe.grouped_gemm_wgrad(self.dgu, self.x, self.off, self.dw13, a_rows=self.rows, a_div=self.k, **kw)
        moe.grouped_gemm_dgrad(self.dgu, self.w13, self.off, self.dxp, out_rows=self.rows, **kw)
        moe.grouped_gemm_w4(self.x[:, :self.K4], self.w4, self.s4, self.off, self.y4, a_rows=self.rows, a_div=self.k,
                            **kw)

    def clear(self):
        for n in self.OUT:
            getattr(self, n).zero_()

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.OUT}


def same(a, b, what):
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), "%s: %s differs" % (what, n)


def test_same_bits_on_side_streams_and_at_once():
    steps = [Step(1), Step(2, M=300, E=4, k=3, H=136, I=264, block=1)]
    alone = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        alone.append(s.outputs())
        s.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for rep in range(3):
        say("two steps at once, round %d" % rep)
        for s, st in zip(steps, streams):
            s.run(st)
        torch.cuda.synchronize()
        for s, a in zip(steps, alone):
            same(a, s.outputs(), "side stream")
            s.clear()
        torch.cuda.synchronize()


def test_outputs_made_for_a_side_stream():
    s = Step(3)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = moe.grouped_gemm(s.x, s.w13, s.off, a_rows=s.rows, a_div=s.k)
    n = int(s.num)
    got = moe.grouped_gemm(s.x, s.w13, s.off, a_rows=s.rows, a_div=s.k, stream=st)
    st.synchronize()
    assert torch.equal(want[:n], got[:n])


def test_captured_and_replayed():
    s = Step(4)
    s.run()
    torch.cuda.synchronize()
    want = s.outputs()
    s.clear()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    other = Step(5)
    for rep in range(4):
        say("replay %d" % rep)
        s.clear()
        g.replay()
        torch.cuda.synchronize()
        same(want, s.outputs(), "replay %d" % rep)
        other.run()  # eager work of the same kernels between the replays
        torch.cuda.synchronize()
    # new inputs in the same buffers
    s.x.copy_(other.x)
    g.replay()
    torch.cuda.synchronize()
    got = s.outputs()
    s.run()
    torch.cuda.synchronize()
    same(s.outputs(), got, "replay on new inputs")


def test_accumulated_weight_gradient():
    s = Step(6)
    s.run()
    once = s.dw13.clone()
    moe.grouped_gemm_wgrad(s.dgu, s.x, s.off, s.dw13, a_rows=s.rows, a_div=s.k, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(s.dw13, once + once)


def test_same_id_twice():
    # input rows may be read by many rows; of two rows written to one place one result stays
    rng = np.random.default_rng(7)
    a, w = bf16(rng, 4, 64), bf16(rng, 2, 72, 64, scale=0.125)
    off = torch.tensor([0, 70, 100], dtype=torch.int32, device=DEV)
    ids = torch.full((100,), 2, dtype=torch.int32, device=DEV)
    y = moe.grouped_gemm(a.to(DEV), w.to(DEV), off, a_rows=ids)
    assert torch.equal(y[:70], y[:1].expand(70, -1)) and torch.equal(y[70:], y[70:71].expand(30, -1))
    out = torch.zeros(3, 72, dtype=torch.bfloat16, device=DEV)
    moe.grouped_gemm(a.to(DEV), w.to(DEV), off, out, a_rows=ids, out_rows=torch.clamp(ids, max=1))
    torch.cuda.synchronize()
    assert not bool(out[0].any()) and not bool(out[2].any())
    assert torch.equal(out[1], y[0]) or torch.equal(out[1], y[70])


@pytest.mark.parametrize("bad", [[-5, 20, 40, 60], [0, 50, 20, 60], [0, 20, 40, 1 << 30], [0, 0, 0, 0],
                                 [60, 40, 20, 0], [-(1 << 31), (1 << 31) - 1, 0, 60]])
def test_offsets_are_clamped(bad):
    # offsets that no routing makes: every access stays inside the R rows, and rows of experts whose own range
    # is sound come out right
    rng = np.random.default_rng(8)
    R, E, N, K = 60, 3, 136, 128
    a, w = bf16(rng, R, K), bf16(rng, E, N, K, scale=K ** -0.5)
    off = torch.tensor(bad, dtype=torch.int64).to(torch.int32).to(DEV)
    full = torch.full((R + 20, N), -7.75, dtype=torch.bfloat16, device=DEV)
    moe.grouped_gemm(a.to(DEV), w.to(DEV), off, full[10:10 + R])
    codes = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)).to(DEV)
    moe.grouped_gemm_w4(a.to(DEV), codes, torch.full((E, N, K // 32), 120, dtype=torch.uint8, device=DEV), off,
                        torch.empty(R, N, dtype=torch.bfloat16, device=DEV))
    dw = moe.grouped_gemm_wgrad(a.to(DEV), a.to(DEV), off)
    torch.cuda.synchronize()
    assert bool((full[:10] == -7.75).all()) and bool((full[10 + R:] == -7.75).all())
    assert bool(torch.isfinite(dw).all())
    lo = np.clip(np.array(bad[:-1], dtype=np.int64), 0, R)
    hi = np.maximum(np.clip(np.array(bad[1:], dtype=np.int64), 0, R), lo)
    for e in range(E):
        alone = [i for i in range(lo[e], hi[e]) if sum(lo[f] <= i < hi[f] for f in range(E)) == 1]
        rows = f64(a)[alone]
        if alone:
            check(full[10:10 + R][torch.tensor(alone, device=DEV)], rows @ f64(w)[e].T, np.abs(rows) @ np.abs(f64(w)[e].T),
                  K, "expert %d" % e)


@pytest.mark.parametrize("fmt,lead", [("mxfp4", 1), ("mxfp4", 2), ("mxfp4", 3), ("int4", 2)])
@pytest.mark.parametrize("K", [128, 384])
def test_scales_at_odd_addresses(fmt, lead, K):
    rng = np.random.default_rng(9)
    E, N, R = 3, 72, 20
    off = offsets_of([9, 0, 11])
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = torch.from_numpy(rng.integers(110, 130, (E, N, K // 32), dtype=np.uint8))
    else:
        scales = torch.from_numpy(rng.uniform(0.01, 0.1, (E, N, K // 128)).astype(np.float32)).to(torch.bfloat16)
    raw = torch.full((scales.numel() * scales.element_size() + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    n = scales.numel() * scales.element_size()
    raw[lead:lead + n] = scales.view(torch.uint8).flatten().to(DEV)
    view = raw[lead:lead + n]
    view = view.view(E, N, K // 32) if fmt == "mxfp4" else view.view(torch.bfloat16).view(E, N, K // 128)
    a = bf16(rng, R, K)
    y = moe.grouped_gemm_w4(a.to(DEV), torch.from_numpy(codes).to(DEV), view, torch.from_numpy(off).to(DEV),
                            out_dtype=torch.float32)
    w = w4_values(codes, scales, fmt)
    mag = np.abs(w) if fmt == "mxfp4" else np.repeat(np.abs(f64(scales)), 128, axis=2) * 55
    for e in range(E):
        s = slice(off[e], off[e + 1])
        check(y[s], f64(a)[s] @ w[e].T, np.abs(f64(a))[s] @ mag[e].T, K, "expert %d" % e)


def test_a_token_is_the_same_in_any_batch():
    # the sums of a row do not depend on the rows around it where the sizes R, E, N, K and its expert's kind of tile
    # are the same: the same rows in another order, other rows' values changed
    rng = np.random.default_rng(10)
    E, N, K = 4, 264, 520
    off = torch.from_numpy(offsets_of([300, 20, 100, 0])).to(DEV)
    a, w = bf16(rng, 420, K).to(DEV), bf16(rng, E, N, K, scale=K ** -0.5).to(DEV)
    y = moe.grouped_gemm(a, w, off)
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(1)).to(DEV)
    b = a.clone()
    b[:300] = a[:300][perm]
    b[300:] = 3.0
    z = moe.grouped_gemm(b, w, off)
    torch.cuda.synchronize()
    assert torch.equal(z[:300], y[:300][perm])


def test_refusals_of_the_binding():
    a = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    ids = torch.arange(8, dtype=torch.int32, device=DEV)
    ok = moe.grouped_gemm(a, w, off)
    assert ok.shape == (8, 32)
    for exc, call in [
        (TypeError, lambda: moe.grouped_gemm(a.float(), w, off)),
        (TypeError, lambda: moe.grouped_gemm(a, w.float(), off)),
        (TypeError, lambda: moe.grouped_gemm(a, w, off.long())),
        (ValueError, lambda: moe.grouped_gemm(a, w, off[:2])),
        (ValueError, lambda: moe.grouped_gemm(a[:, :56], w, off)),
        (ValueError, lambda: moe.grouped_gemm(a.t(), w, off)),
        (ValueError, lambda: moe.grouped_gemm(a, w.transpose(1, 2), off)),
        (ValueError, lambda: moe.grouped_gemm(a, w[0], off)),
        (TypeError, lambda: moe.grouped_gemm(a, w, off, out_dtype=torch.float16)),
        (ValueError, lambda: moe.grouped_gemm(a, w, off, torch.zeros(8, 40, dtype=torch.bfloat16, device=DEV))),
        (ValueError, lambda: moe.grouped_gemm(a, w, off, out_rows=ids[:5])),
        (TypeError, lambda: moe.grouped_gemm(a, w, off, a_rows=ids.long())),
        (moe.MoEError, lambda: moe.grouped_gemm(a, w, off, a_rows=ids, a_div=0)),
        (moe.MoEError, lambda: moe.grouped_gemm(a, w, off, torch.zeros(7, 32, dtype=torch.bfloat16, device=DEV))),
        (ValueError, lambda: moe.grouped_gemm(a, w.cpu(), off)),
        (ValueError, lambda: moe.grouped_gemm_wgrad(a, a, off, accumulate=True)),
        (moe.MoEError, lambda: moe.grouped_gemm_wgrad(
            a, a, off, torch.zeros(2, 64, 64, dtype=torch.bfloat16, device=DEV), accumulate=True)),
        (ValueError, lambda: moe.grouped_gemm_w4(
            a, torch.zeros(2, 32, 32, dtype=torch.uint8, device=DEV), torch.zeros(2, 32, 1, dtype=torch.uint8, device=DEV),
            off)),
        (moe.MoEError, lambda: moe.grouped_gemm_w4(
            a[:, :48], torch.zeros(2, 32, 24, dtype=torch.uint8, device=DEV),
            torch.zeros(2, 32, 1, dtype=torch.uint8, device=DEV), off)),
        (ValueError, lambda: moe.swiglu_checkpoint(a[:, :63])),
        (ValueError, lambda: moe.swiglu_checkpoint(a, row_weight=torch.ones(7, device=DEV))),
        (ValueError, lambda: moe.swiglu_checkpoint(a, checkpoint=False, codes=a.view(torch.uint8))),
        (moe.MoEError, lambda: moe.swiglu_checkpoint(torch.zeros(4, 24, dtype=torch.bfloat16, device=DEV))),
    ]:
        with pytest.raises(exc):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gather_dy,gather_a", [(True, False), (False, True), (True, True)])
def test_masked_rows_add_nothing(gather_dy, gather_a, dtype):
    # a row that an id masks in one operand may hold anything in the other
    say("wgrad masked rows gather=%s,%s %s" % (gather_dy, gather_a, dtype))
    rng = np.random.default_rng(10)
    counts, N, K = [70, 1, 0, 333], 264, 136
    off, R = offsets_of(counts), sum(counts)
    kinds = [k for k, g in (("dy", gather_dy), ("a", gather_a)) if g]
    masked = {k: rng.random(R) < 0.2 for k in kinds}
    masked[kinds[0]][70] = True  # an expert whose only row is masked
    masked[kinds[0]][404 - 64:] = True  # and a whole step
    hidden = np.logical_or.reduce([masked[k] for k in kinds])
    ops, ids, sums = {}, {}, {}
    for k, width in (("dy", N), ("a", K)):
        rows = bf16(rng, R, width)
        t = rows.clone()
        t[torch.from_numpy(hidden)] = torch.tensor([float("nan"), float("inf")], dtype=t.dtype).repeat(width // 2)
        sums[k] = np.where(hidden[:, None], 0.0, f64(rows))
        ids[k] = None
        if k in kinds:
            perm = rng.permutation(R)
            where = np.argsort(perm).astype(np.int32)
            t = t[torch.from_numpy(perm)]
            where[masked[k]] = np.where(rng.random(masked[k].sum()) < 0.5, -1, R)
            ids[k] = torch.from_numpy(where).to(DEV)
        ops[k] = t.to(DEV)
    got = moe.grouped_gemm_wgrad(ops["dy"], ops["a"], torch.from_numpy(off).to(DEV), dy_rows=ids["dy"],
                                 a_rows=ids["a"], out_dtype=dtype)
    torch.cuda.synchronize()
    for e, n in enumerate(counts):
        x, y = sums["dy"][off[e]:off[e + 1]], sums["a"][off[e]:off[e + 1]]
        check(got[e], x.T @ y, np.abs(x).T @ np.abs(y), n, "expert %d" % e)
