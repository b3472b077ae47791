"""The gated activation with its 8-bit checkpoint, and its gradient, on the
GPU against the definitions in 64 bits; the gradient also against differences;
and a training step of a layer's expert half, end to end."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import BF16_STEP, DEV, Canvas, bf16, f64

pytestmark = pytest.mark.gpu

E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8.0 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where(c >= 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


def scale_codes(v: np.ndarray) -> np.ndarray:
    """E8M0 codes of float64 groups [..., 32]: the smallest power of two under
    which the largest finite magnitude does not pass 448, at least 2^-127."""
    top = np.where(np.isfinite(v), np.abs(v), 0.0).max(-1)
    m, ex = np.frexp(top / E4M3_MAX)  # top/448 = m * 2^ex, m in [0.5, 1)
    return np.where(top > 0, np.maximum(np.where(m == 0.5, ex - 1, ex) + 127, 0), 0)


def groups_of(half: np.ndarray) -> np.ndarray:
    R, I = half.shape
    G = -(-I // 32)
    full = np.zeros((R, G * 32))
    full[:, :I] = half
    return full.reshape(R, G, 32)


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 [R, 2, I] of a checkpoint."""
    R, I = codes.shape[0], codes.shape[1] // 2
    s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=2)[:, :, :I]
    return e4m3_values()[codes].reshape(R, 2, I) * s


def sigmoid(g):
    return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def inputs(R, I, seed, spread=2.0):
    rng = np.random.default_rng([seed, R, I])
    gu = rng.standard_normal((R, 2 * I)) * np.exp(spread * rng.standard_normal((R, 1)))
    gu[:, ::37] *= 1e-3
    gu[:, I // 2] *= 30
    return rng, torch.from_numpy(gu.astype(np.float32)).to(torch.bfloat16)


# h = w SiLU(g) u: an exp2 and a reciprocal of about an ulp and four products in fp32, 2^-20 in all, then the bf16
# step.  exp2's argument is rounded at |g|*2^-24*1.45, a relative error of the exponential that is at most g*2^-23 of
# it where it matters (|g| < 90), hence the |g| term.  Below g = -87.3 the sigmoid is smaller than 2^-126, the least
# normal fp32: exp(-g) overflows or its reciprocal is flushed, and the sigmoid comes out as 0, an absolute error of up
# to 2^-126, which `outer`, the product of the other factors, multiplies.
def h_bound(ref, g, outer):
    rel = 2.0 ** -20 + np.minimum(np.abs(g), 90) * 2.0 ** -23
    return np.abs(ref) * (BF16_STEP * (1 + rel) + rel) + 2.0 ** -126 * (1 + np.abs(outer))


SHAPES = [(1, 8), (3, 24), (5, 32), (2, 40), (7, 264), (33, 768), (4, 1544), (2, 4104), (130, 96)]


@pytest.mark.parametrize("R,I", SHAPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_checkpoint(R, I, weighted):
    say("checkpoint R=%d I=%d weighted=%s" % (R, I, weighted))
    rng, gu = inputs(R, I, 1)
    w = torch.from_numpy(rng.uniform(-1, 2, R).astype(np.float32)) if weighted else None
    G = -(-I // 32)
    codes = torch.full((R + 2, 2 * I), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((R + 2, 2, G), 0xAB, dtype=torch.uint8, device=DEV)
    h = torch.full((R + 2, I), -7.75, dtype=torch.bfloat16, device=DEV)
    full = torch.full((R, 2 * I + 16), float("nan"), dtype=torch.bfloat16, device=DEV)
    full[:, :2 * I] = gu.to(DEV)
    moe.swiglu_checkpoint(full[:, :2 * I], None if w is None else w.to(DEV), h=h[1:R + 1], codes=codes[1:R + 1],
                          scales=scales[1:R + 1])
    torch.cuda.synchronize()
    for t, m in ((codes, 0xAB), (scales, 0xAB), (h, -7.75)):
        assert bool((t[0] == m).all()) and bool((t[R + 1] == m).all())
    v = f64(gu).reshape(R, 2, I)
    ref = v[:, 0] * sigmoid(v[:, 0]) * v[:, 1] * (1.0 if w is None else f64(w)[:, None])
    outer = v[:, 0] * v[:, 1] * (1.0 if w is None else f64(w)[:, None])
    ok = np.abs(f64(h[1:R + 1]) - ref) <= h_bound(ref, v[:, 0], outer)
    assert ok.all(), (v[:, 0][~ok][:4], v[:, 1][~ok][:4], ref[~ok][:4], f64(h[1:R + 1])[~ok][:4])
    want = np.stack([scale_codes(groups_of(v[:, k])) for k in (0, 1)], 1)
    got = scales[1:R + 1].cpu().numpy()
    assert np.array_equal(got, want)
    dec = decode(codes[1:R + 1].cpu().numpy(), got)
    s = np.repeat(2.0 ** (got.astype(np.float64) - 127), 32, axis=2)[:, :, :I]
    # half a step of the value's binade, or of the subnormal grid 2^-9
    half = np.maximum(np.abs(v) * 2.0 ** -4, s * 2.0 ** -10)
    assert (np.abs(dec - v) <= half).all()
    # nearest: no other code is nearer, and ties take the even code
    grid = np.sort(np.unique(e4m3_values()[~np.isnan(e4m3_values())]))
    q = (v / s).ravel()
    near = np.abs(grid[np.clip(np.searchsorted(grid, q)[:, None] + np.arange(-1, 1), 0, grid.size - 1)] - q[:, None])
    assert np.array_equal(np.abs(dec / s - v / s).ravel(), near.min(1))
    tie = near[:, 0] == near[:, 1]
    assert not (codes[1:R + 1].cpu().numpy().reshape(R, 2, I).ravel()[tie] & 1).any()


def test_checkpoint_special_values():
    # every finite bf16 magnitude as the largest of its group, and what is not finite
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    R = v.numel()
    gu = torch.zeros(R, 64, dtype=torch.bfloat16)
    gu[:, 0] = v
    gu[:, 33] = -v
    gu[:, 34] = v / 4
    h, codes, scales = moe.swiglu_checkpoint(gu.to(DEV))
    x = f64(gu).reshape(R, 2, 32)
    want = scale_codes(x)
    assert np.array_equal(scales.cpu().numpy()[:, :, 0], want)
    dec = decode(codes.cpu().numpy(), scales.cpu().numpy())
    s = 2.0 ** (want.astype(np.float64) - 127)[:, :, None]
    assert (np.abs(dec - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)).all()
    assert (np.abs(dec / s).max(-1) <= E4M3_MAX).all()
    gu = torch.ones(3, 64, dtype=torch.bfloat16)
    gu[0, 3], gu[1, 40], gu[2, 5] = float("nan"), float("inf"), -float("inf")
    _, codes, scales = moe.swiglu_checkpoint(gu.to(DEV))
    c, dec = codes.cpu().numpy(), decode(codes.cpu().numpy(), scales.cpu().numpy()).reshape(3, 64)
    where = np.zeros((3, 64), dtype=bool)
    where[0, 3] = where[1, 40] = where[2, 5] = True
    assert (c[where] == 0x7F).all() and (dec[~where] == 1.0).all()


def grad_reference(dec, dh, w):
    g, u = dec[:, 0], dec[:, 1]
    s = sigmoid(g)
    d = dh * w[:, None]
    return d * u * s * (1 + g * sigmoid(-g)), d * g * s, w[:, None] * g * s * u, g * s * u * dh


@pytest.mark.parametrize("R,I", SHAPES + [(600, 8), (9, 2056), (2, 8200)])
@pytest.mark.parametrize("weighted", [False, True])
def test_grad(R, I, weighted):
    say("checkpoint grad R=%d I=%d weighted=%s" % (R, I, weighted))
    rng, gu = inputs(R, I, 2, 1.0)
    _, codes, scales = moe.swiglu_checkpoint(gu.to(DEV))
    dh = bf16(rng, R, I)
    w = torch.from_numpy(rng.uniform(-1, 2, R).astype(np.float32)) if weighted else None
    dgu, h = Canvas(R, 2 * I, torch.bfloat16, pad_cols=0), Canvas(R, I, torch.bfloat16, pad_cols=0)
    dwt = torch.full((R + 2,), -7.75, device=DEV)
    moe.swiglu_checkpoint_grad(codes, scales, dh.to(DEV), None if w is None else w.to(DEV), dgu=dgu.t, h=h.t,
                               dweight=dwt[1:R + 1])
    torch.cuda.synchronize()
    for c in (dgu, h):
        c.check_untouched(np.ones(R, dtype=bool))
    assert float(dwt[0]) == -7.75 and float(dwt[R + 1]) == -7.75
    dec = decode(codes.cpu().numpy(), scales.cpu().numpy())
    dg, du, hr, terms = grad_reference(dec, f64(dh), f64(w) if weighted else np.ones(R))
    g = np.abs(dec[:, 0])
    got = f64(dgu.t)
    wd = f64(dh) * (f64(w)[:, None] if weighted else 1.0)
    ok_h = np.abs(f64(h.t) - hr) <= h_bound(hr, g, dec[:, 0] * dec[:, 1])
    assert ok_h.all(), (np.argwhere(~ok_h)[:4], hr[~ok_h][:4], f64(h.t)[~ok_h][:4])
    ok_u = np.abs(got[:, I:] - du) <= h_bound(du, g, wd * dec[:, 0])
    assert ok_u.all(), (np.argwhere(~ok_u)[:4], du[~ok_u][:4], got[:, I:][~ok_u][:4])
    # 1 + g(1-s): 1 - s is off by 2^-24 and multiplied by g, so the bracket by g*2^-23 + 2^-23; the factor outside it as above
    d = np.abs(wd * dec[:, 1]) * sigmoid(dec[:, 0])
    extra = d * (g + 2) * 2.0 ** -21
    ok_g = np.abs(got[:, :I] - dg) <= h_bound(dg, g, wd * dec[:, 1] * (1 + g)) + extra * (1 + BF16_STEP)
    assert ok_g.all(), (np.argwhere(~ok_g)[:4], dg[~ok_g][:4], got[:, :I][~ok_g][:4])
    sums = np.abs(terms)
    tol = (sums * (2.0 ** -20 + np.minimum(g, 90) * 2.0 ** -23)).sum(1) + (I + 16) * 2.0 ** -24 * sums.sum(1)
    assert (np.abs(f64(dwt[1:R + 1]) - terms.sum(1)) <= tol + 1e-30).all(), \
        (f64(dwt[1:R + 1]) - terms.sum(1), tol)


def test_grad_matches_differences():
    # values on the checkpoint's grid, so that it stands for them exactly: the op's gradient against central
    # differences of the definition in 64 bits
    R, I = 6, 96
    rng = np.random.default_rng(5)
    grid = e4m3_values()
    ok = np.nonzero(~np.isnan(grid) & (np.abs(grid) <= 6) & (np.abs(grid) >= 2.0 ** -5))[0]
    gu = torch.from_numpy(grid[rng.choice(ok, (R, 2 * I))].astype(np.float32)).to(torch.bfloat16)
    gu[:, ::32] = 6.0  # one scale for every group, well above the grid's subnormals
    w = torch.from_numpy(rng.uniform(0.2, 1, R).astype(np.float32))
    dh = bf16(rng, R, I)
    _, codes, scales = moe.swiglu_checkpoint(gu.to(DEV), w.to(DEV))
    assert np.array_equal(decode(codes.cpu().numpy(), scales.cpu().numpy()).reshape(R, 2 * I), f64(gu))
    dgu, _, dwt = moe.swiglu_checkpoint_grad(codes, scales, dh.to(DEV), w.to(DEV))

    def loss(x, ww):
        return (ww[:, None] * x[:, :I] * sigmoid(x[:, :I]) * x[:, I:] * f64(dh)).sum(1)

    x, eps = f64(gu), 1e-5
    got = f64(dgu)
    for col in range(0, 2 * I, 5):
        dx = np.zeros_like(x)
        dx[:, col] = eps
        diff = (loss(x + dx, f64(w)) - loss(x - dx, f64(w))) / (2 * eps)
        # a central difference is off by eps^2/6 times a third derivative below 40, and by its sums' rounding over eps
        assert (np.abs(got[:, col] - diff) <= np.abs(diff) * (BF16_STEP + 2.0 ** -18) + 1e-5).all()
    diff = (loss(x, f64(w) + eps) - loss(x, f64(w) - eps)) / (2 * eps)
    assert (np.abs(f64(dwt) - diff) <= 1e-4 * np.abs(f64(dh)).sum(1)).all()


def test_num_rows():
    R, I, n = 40, 72, 17
    rng, gu = inputs(R, I, 4)
    gu[n:] = float("nan")
    num = torch.tensor([n], dtype=torch.int32, device=DEV)
    h = torch.full((R, I), -7.75, dtype=torch.bfloat16, device=DEV)
    codes = torch.full((R, 2 * I), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((R, 2, 3), 0xAB, dtype=torch.uint8, device=DEV)
    moe.swiglu_checkpoint(gu.to(DEV), num_rows=num, h=h, codes=codes, scales=scales)
    want = moe.swiglu_checkpoint(gu[:n].to(DEV))
    for got, ref, mark in zip((h, codes, scales), want, (-7.75, 0xAB, 0xAB)):
        assert torch.equal(got[:n], ref) and bool((got[n:] == mark).all())
    dh = bf16(rng, R, I).to(DEV)
    dgu = torch.full((R, 2 * I), -7.75, dtype=torch.bfloat16, device=DEV)
    h2 = torch.full((R, I), -7.75, dtype=torch.bfloat16, device=DEV)
    dwt = torch.full((R,), -7.75, device=DEV)
    moe.swiglu_checkpoint_grad(codes, scales, dh, num_rows=num, dgu=dgu, h=h2, dweight=dwt)
    want = moe.swiglu_checkpoint_grad(codes[:n], scales[:n], dh[:n])
    for got, ref in zip((dgu, h2, dwt), want):
        assert torch.equal(got[:n], ref) and bool((got[n:] == -7.75).all())


def test_activation_alone():
    _, gu = inputs(9, 264, 6)
    h, codes, scales = moe.swiglu_checkpoint(gu.to(DEV), checkpoint=False)
    assert codes is None and scales is None
    assert torch.equal(h, moe.swiglu_checkpoint(gu.to(DEV))[0])


def test_empty():
    h, codes, scales = moe.swiglu_checkpoint(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert h.shape == (0, 32) and codes.shape == (0, 64) and scales.shape == (0, 2, 1)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    a = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(3, 32, 64, dtype=torch.bfloat16, device=DEV)
    assert moe.grouped_gemm(a, w, off).shape == (0, 32)
    dw = moe.grouped_gemm_wgrad(torch.empty(0, 32, dtype=torch.bfloat16, device=DEV), a, off)
    assert dw.shape == (3, 32, 64) and not bool(dw.any())


@pytest.mark.parametrize("block,M,E,k,H,I", [(1, 37, 5, 2, 136, 72), (16, 200, 8, 3, 256, 136), (128, 300, 4, 2, 128, 264)])
def test_training_step(block, M, E, k, H, I):
    """Routing, gathered gate/up product, checkpointed activation, down product
    scattered to pair order; then the gradients of the hidden states, both
    weights and the routing weights, each against the step's formula in 64
    bits on the values the step before it produced."""
    say("training step block=%d M=%d E=%d k=%d H=%d I=%d" % (block, M, E, k, H, I))
    rng = np.random.default_rng([block, M])
    x, dy = bf16(rng, M, H), bf16(rng, M, H)
    w13, w2 = bf16(rng, E, 2 * I, H, scale=H ** -0.5), bf16(rng, E, H, I, scale=I ** -0.5)
    logits = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32))
    xd, dyd, w13d, w2d = (t.to(DEV) for t in (x, dy, w13, w2))
    P = M * k
    ids, wts = moe.route_topk(logits.to(DEV), k)
    al = moe.align(ids, E, block)
    off, srt = al["offsets"], al["sorted_ids"]
    num = off[E:]
    R = srt.numel()
    n = int(num[0])
    gu = moe.grouped_gemm(xd, w13d, off, a_rows=srt, a_div=k)
    srt_n = srt[:n].cpu().numpy()
    real = srt_n < P
    rw = torch.zeros(R, device=DEV)
    rw[:n][torch.from_numpy(real).to(DEV)] = wts.flatten()[srt[:n][torch.from_numpy(real).to(DEV)].long()]
    h, codes, scales = moe.swiglu_checkpoint(gu, rw, num_rows=num)
    o = moe.grouped_gemm(h, w2d, off, torch.zeros(P, H, dtype=torch.bfloat16, device=DEV), out_rows=srt)
    y = o.view(M, k, H).float().sum(1)
    # backward
    dh = moe.grouped_gemm_dgrad(dyd, w2d, off, dy_rows=srt, dy_div=k)
    dgu, hw, dwt = moe.swiglu_checkpoint_grad(codes, scales, dh, rw, num_rows=num)
    dw2 = moe.grouped_gemm_wgrad(dyd, hw, off, dy_rows=srt, dy_div=k)
    dw13 = moe.grouped_gemm_wgrad(dgu, xd, off, a_rows=srt, a_div=k)
    dxp = moe.grouped_gemm_dgrad(dgu, w13d, off, torch.zeros(P, H, dtype=torch.bfloat16, device=DEV), out_rows=srt)
    dx = dxp.view(M, k, H).float().sum(1)
    torch.cuda.synchronize()

    # the layer's formula in 64 bits, end to end; the gate and up values that the backward pass uses are those the
    # checkpoint stands for
    X, DY, W13, W2 = f64(x), f64(dy), f64(w13), f64(w2)
    e_of, wt = ids.cpu().numpy(), f64(wts)
    Y, DX = np.zeros((M, H)), np.zeros((M, H))
    DW13, DW2, DWT = np.zeros(W13.shape), np.zeros(W2.shape), np.zeros((M, k))
    kept = decode(codes[:n].cpu().numpy(), scales[:n].cpu().numpy())
    pos = np.full(P, -1)
    pos[srt_n[real]] = np.nonzero(real)[0]
    for m in range(M):
        for j in range(k):
            e = e_of[m, j]
            gv = W13[e] @ X[m]
            g, u = gv[:I], gv[I:]
            Y[m] += wt[m, j] * (W2[e] @ (g * sigmoid(g) * u))
            g, u = kept[pos[m * k + j]]
            s = sigmoid(g)
            hh = g * s * u
            dhh = W2[e].T @ DY[m]
            DWT[m, j] = dhh @ hh
            DW2[e] += np.outer(DY[m], wt[m, j] * hh)
            d = np.concatenate([dhh * u * s * (1 + g * (1 - s)), dhh * g * s]) * wt[m, j]
            DW13[e] += np.outer(d, X[m])
            DX[m] += W13[e].T @ d
    got_wt = np.zeros((M, k))
    got_wt.reshape(-1)[srt_n[real]] = f64(dwt[:n])[real]

    # Each product's operands were rounded to bf16 up to three times on the way (gu, h, o; dh, dgu, dx): half a step
    # each, 2^-8 of a value at most, random in sign, so the norm of a result is off by at most 3 * 2^-8 of its own
    # (gu's rounding passes through SiLU(g)*u, whose relative condition is 1 + |g|(1-s) + 1, on average below 3)
    def near(got, ref, steps, what):
        err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        say("  %s: %.2e" % (what, err))
        assert err <= steps * BF16_STEP, (what, err)

    near(f64(y), Y, 5, "y")
    near(f64(dx), DX, 3, "dx")
    near(f64(dw13), DW13, 2, "dw13")
    near(f64(dw2), DW2, 1, "dw2")
    near(got_wt, DWT, 1, "dweight")


@pytest.mark.parametrize("R", [(1 << 26) - 1, (1 << 26) - 3, (1 << 26) - 4])
def test_most_rows(R):
    # the most rows there may be, of the shortest length: a grid of 2^32 threads
    say("checkpoint and gradient of %d rows" % R)
    I, n = 8, 4096
    rng, gu = inputs(n, I, 8, 1.0)
    gu, dh, wt = gu.to(DEV), bf16(rng, n, I).to(DEV), torch.from_numpy(rng.uniform(0.2, 1, n).astype(np.float32)).to(DEV)
    reps = -(-R // n)
    want = moe.swiglu_checkpoint(gu, wt)
    got = moe.swiglu_checkpoint(gu.repeat(reps, 1)[:R], wt.repeat(reps)[:R])
    for g, w in zip(got, want):
        for lo in (0, R // 2 // n * n, R // n * n - n, R // n * n):
            m = min(n, R - lo)
            assert torch.equal(g[lo:lo + m], w[:m])
    del got
    want = moe.swiglu_checkpoint_grad(want[1], want[2], dh, wt)
    _, codes, scales = moe.swiglu_checkpoint(gu)
    got = moe.swiglu_checkpoint_grad(codes.repeat(reps, 1)[:R], scales.repeat(reps, 1, 1)[:R], dh.repeat(reps, 1)[:R],
                                     wt.repeat(reps)[:R])
    for g, w in zip(got, want):
        for lo in (0, R // 2 // n * n, R // n * n - n, R // n * n):
            m = min(n, R - lo)
            assert torch.equal(g[lo:lo + m], w[:m])


def test_most_groups():
    # a bound of almost 2^30 rows times groups, of which the device's own count leaves five rows
    I, G, n = 544, 17, 5
    R = ((1 << 30) - 1) // G
    say("checkpoint and gradient of at most %d rows of %d" % (R, I))
    rng, gu = inputs(n, I, 9, 1.0)
    gu, dh = gu.to(DEV), bf16(rng, n, I).to(DEV)
    num = torch.tensor([n], dtype=torch.int32, device=DEV)
    h, codes, scales = (torch.zeros(s, dtype=t, device=DEV) for s, t in (
        ((n, I), torch.bfloat16), ((n, 2 * I), torch.uint8), ((n, 2, G), torch.uint8)))
    lib = moe.load()
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.moe_swiglu_checkpoint(gu.data_ptr(), 2 * I, None, R, I, num.data_ptr(), h.data_ptr(), codes.data_ptr(),
                                     scales.data_ptr(), stream) == 0
    for g, w in zip((h, codes, scales), moe.swiglu_checkpoint(gu)):
        assert torch.equal(g, w)
    dgu, hw = torch.zeros(n, 2 * I, dtype=torch.bfloat16, device=DEV), torch.zeros_like(h)
    dwt = torch.zeros(n, device=DEV)
    assert lib.moe_swiglu_checkpoint_grad(codes.data_ptr(), scales.data_ptr(), dh.data_ptr(), None, R, I, num.data_ptr(),
                                          dgu.data_ptr(), hw.data_ptr(), dwt.data_ptr(), stream) == 0
    for g, w in zip((dgu, hw, dwt), moe.swiglu_checkpoint_grad(codes, scales, dh)):
        assert torch.equal(g, w)
