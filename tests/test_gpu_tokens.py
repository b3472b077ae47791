"""The tokens' way to their experts and back on the GPU, with its gradients and
the router's, against plain loops and sums in 64 bits: dropped pairs, tokens and
experts without pairs, experts of other processes, equal ids, odd sizes, strides,
poisoned surroundings, every way of counting the pairs; and a training step of
all of it together."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import BF16_STEP, DEV, Canvas, bf16, check, f64, poisoned, sum_bound

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def routing(rng, M, k, E, first=0, drop=0.0, skew=0.0, equal=False):
    """int32 ids [M,k] with experts outside [first, first+E) among them."""
    score = rng.standard_normal((M, E + 2 * first)) - skew * np.log1p(np.arange(E + 2 * first))
    if equal:
        ids = rng.integers(0, E + 2 * first, (M, k))
    else:
        ids = np.argsort(-score, axis=1, kind="stable")[:, :k]
    ids = ids.astype(np.int32)
    ids[rng.random((M, k)) < drop] = -1
    if drop:
        ids[rng.random((M, k)) < drop / 4] = np.iinfo(np.int32).max
        ids[rng.random((M, k)) < drop / 4] = np.iinfo(np.int32).min
        ids[: M // 5] = -1  # tokens of the padding
    return ids


def layout(ids, E, first=0):
    """(offsets, positions, pairs) by plain loops."""
    held = [[] for _ in range(E)]
    for f, e in enumerate(ids.reshape(-1).tolist()):
        if first <= e < first + E:
            held[e - first].append(f)
    pairs = np.array([f for h in held for f in h], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(h) for h in held])])
    positions = np.full(ids.size, -1)
    positions[pairs] = np.arange(len(pairs))
    return offsets, positions.reshape(ids.shape), np.concatenate([pairs, np.full(ids.size - len(pairs), -1)])


def check_dispatch(x, ids, E, first, dtype=torch.bfloat16, pad=8):
    M, k = ids.shape
    H = x.shape[1]
    canvas = Canvas(M * k, H, torch.float32 if dtype not in Canvas.MARK else dtype, pad_cols=pad)
    out = canvas.t
    got, off, pos, pairs = moe.dispatch(x, torch.from_numpy(ids).to(DEV), E, out, first_expert=first)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    r_off, r_pos, r_pairs = layout(ids, E, first)
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(pos.cpu().numpy(), r_pos)
    assert np.array_equal(pairs.cpu().numpy(), r_pairs)
    n = r_off[-1]
    written = np.zeros(M * k, dtype=bool)
    written[:n] = True
    canvas.check_untouched(written)
    token = torch.from_numpy(r_pairs[:n] // k).to(DEV)
    assert torch.equal(out[:n], x[token])
    # the layout alone
    none, *alone = moe.dispatch(None, torch.from_numpy(ids).to(DEV), E, first_expert=first)
    assert none is None and all(torch.equal(a, b) for a, b in zip(alone, (off, pos, pairs)))


# the pairs counted by every workgroup (up to 4096), as sums of chunks, and scanned
SHAPES = [(1, 1, 1), (1, 2, 8), (3, 16, 16), (33, 8, 128), (77, 3, 7), (511, 8, 512), (512, 8, 128), (4096, 1, 5),
          (513, 8, 8), (1500, 3, 130), (1025, 16, 17), (2500, 8, 512), (9000, 2, 257)]


@pytest.mark.parametrize("M,k,E", SHAPES)
@pytest.mark.parametrize("kind", ["plain", "dropped", "share"])
def test_dispatch(M, k, E, kind):
    say("dispatch M=%d k=%d E=%d %s" % (M, k, E, kind))
    rng = np.random.default_rng([M, k, E])
    first = 3 if kind == "share" else 0
    ids = routing(rng, M, k, E, first, 0.2 if kind == "dropped" else 0.0, 1.0, kind == "share")
    H = 72 if M > 600 else 264
    check_dispatch(poisoned(bf16(rng, M, H), 8), ids, E, first)


@pytest.mark.parametrize("M,k,E", [(5, 2, 4), (700, 8, 32)])
@pytest.mark.parametrize("what", ["none", "one", "same"])
def test_dispatch_uneven(M, k, E, what):
    # nothing held; one pair in all; every pair with the same expert
    ids = np.full((M, k), E if what != "same" else E - 1, dtype=np.int32)
    if what == "one":
        ids[M // 2, k - 1] = 2
    rng = np.random.default_rng(1)
    check_dispatch(bf16(rng, M, 8).to(DEV), ids, E, 0)


@pytest.mark.parametrize("M,H", [(1, 8), (1, 2056), (2, 8192), (17, 4096), (300, 1032)])
def test_dispatch_widths(M, H):
    # few tokens: workgroups share their rows
    rng = np.random.default_rng([M, H])
    check_dispatch(bf16(rng, M, H).to(DEV), routing(rng, M, 4, 9), 9, 0)


@pytest.mark.parametrize("dtype,H", [(torch.int8, 48), (torch.uint8, 1040), (torch.float16, 24), (torch.float32, 20)])
def test_dispatch_types(dtype, H):
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.integers(-100, 100, (50, H))).to(dtype).to(DEV)
    ids = routing(rng, 50, 3, 10, drop=0.1)
    rows, off, pos, pairs = moe.dispatch(x, torch.from_numpy(ids).to(DEV), 10)
    r_off, r_pos, r_pairs = layout(ids, 10)
    n = r_off[-1]
    assert np.array_equal(pos.cpu().numpy(), r_pos)
    assert torch.equal(rows[:n], x[torch.from_numpy(r_pairs[:n] // 3).to(DEV)])


def test_no_tokens():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    rows, off, pos, pairs = moe.dispatch(x, torch.empty(0, 2, dtype=torch.int32, device=DEV), 5)
    assert rows.shape == (0, 64) and off.tolist() == [0] * 6 and pos.shape == (0, 2) and pairs.shape == (0,)
    w = torch.empty(0, 2, device=DEV)
    assert moe.combine(rows, pos, w).shape == (0, 64)
    assert [t.shape for t in moe.combine_grad(x, rows, pos, w)] == [(0, 64), (0, 2)]
    assert moe.route_topk_grad(pos, w, w, 5).shape == (0, 5)
    # tokens, but no rows at all
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    assert not bool(moe.combine(rows, none, torch.full((3, 2), float("nan"), device=DEV)).any())


def combine_case(M, k, E, H, rows_type, y_type, weighted, drop, seed=0):
    """Inputs of a combine: rows with NaN where no position leads, NaN weights of slots without a row."""
    rng = np.random.default_rng([seed, M, k, E, H])
    ids = routing(rng, M, k, E, drop=drop, skew=0.5)
    off, pos, _ = layout(ids, E)
    R, n = M * k, off[-1]
    rows = torch.from_numpy(rng.standard_normal((R, H)).astype(np.float32)).to(TYPES[rows_type])
    rows[n:] = float("nan")
    pos = pos.astype(np.int32)
    if drop:
        pos[(pos < 0) & (rng.random(pos.shape) < 0.5)] = R  # past the rows: no row either
    w = rng.random((M, k)).astype(np.float32) - 0.2
    valid = (pos >= 0) & (pos < R)
    w[~valid] = np.nan
    return rng, rows, pos, valid, (w if weighted else None)


CASES = [(1, 1, 1, 8), (1, 2, 8, 4096), (5, 16, 16, 2064), (64, 8, 32, 2048), (77, 3, 7, 520), (300, 4, 9, 72),
         (130, 6, 64, 1032), (9, 2, 4, 14336), (40, 5, 12, 200), (33, 16, 16, 64), (50, 3, 8, 256), (600, 8, 8, 128),
         (21, 9, 30, 24)]


@pytest.mark.parametrize("M,k,E,H", CASES)
@pytest.mark.parametrize("rows_type,y_type", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("weighted,drop", [(True, 0.0), (True, 0.3), (False, 0.3)])
def test_combine(M, k, E, H, rows_type, y_type, weighted, drop):
    say("combine %s %s" % ((M, k, E, H), (rows_type, y_type, weighted, drop)))
    rng, rows, pos, valid, w = combine_case(M, k, E, H, rows_type, y_type, weighted, drop)
    canvas = Canvas(M, H, TYPES[y_type])
    got = moe.combine(poisoned(rows, 8), torch.from_numpy(pos).to(DEV),
                      None if w is None else torch.from_numpy(w).to(DEV), canvas.t)
    torch.cuda.synchronize()
    assert got.data_ptr() == canvas.t.data_ptr()
    canvas.check_untouched(np.ones(M, dtype=bool))
    wt = np.where(valid, 1.0 if w is None else np.nan_to_num(w).astype(np.float64), 0.0)
    r = np.nan_to_num(f64(rows))[np.where(valid, pos, 0)]
    check(canvas.t, (wt[:, :, None] * r).sum(1), (np.abs(wt)[:, :, None] * np.abs(r)).sum(1), k, "combine")


@pytest.mark.parametrize("M,k,E,H", CASES)
@pytest.mark.parametrize("dy_type,rows_type,out", [("bf16", "bf16", "bf16"), ("fp32", "bf16", "fp32"),
                                                   ("bf16", "fp32", "bf16"), ("fp32", "fp32", "fp32")])
@pytest.mark.parametrize("weighted,drop", [(True, 0.0), (True, 0.3), (False, 0.3)])
def test_combine_grad(M, k, E, H, dy_type, rows_type, out, weighted, drop):
    say("combine_grad %s %s" % ((M, k, E, H), (dy_type, rows_type, out, weighted, drop)))
    rng, rows, pos, valid, w = combine_case(M, k, E, H, rows_type, out, weighted, drop, 1)
    R = M * k
    dy = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(TYPES[dy_type])
    canvas = Canvas(R, H, TYPES[out])
    tp = torch.from_numpy(pos).to(DEV)
    tw = None if w is None else torch.from_numpy(w).to(DEV)
    drows, dw = moe.combine_grad(poisoned(dy, 8), poisoned(rows, 16), tp, tw, canvas.t)
    torch.cuda.synchronize()
    written = np.zeros(R, dtype=bool)
    written[pos[valid]] = True
    canvas.check_untouched(written)
    wt = np.where(valid, 1.0 if w is None else np.nan_to_num(w).astype(np.float64), 0.0)
    ref = wt[:, :, None] * f64(dy)[:, None, :]
    g = f64(canvas.t)[pos[valid]]
    # one rounding in fp32, one to the type
    tol = (2.0 ** -24 + (BF16_STEP if out == "bf16" else 0.0)) * 1.01
    assert (np.abs(g - ref[valid]) <= tol * np.abs(ref[valid]) + 1e-30).all()
    r = np.nan_to_num(f64(rows))[np.where(valid, pos, 0)] * valid[:, :, None]
    terms = r * f64(dy)[:, None, :]
    check(dw, terms.sum(2), np.abs(terms).sum(2), H, "dweights")
    assert not bool(dw.cpu()[torch.from_numpy(~valid)].any())
    # each of the two alone: the same bits
    only, none = moe.combine_grad(dy.to(DEV), None, tp, tw, num_rows=R, out_dtype=TYPES[out])
    assert none is None and torch.equal(only[torch.from_numpy(written)], canvas.t[torch.from_numpy(written)])


@pytest.mark.parametrize("M,k,H,drop", [(13001, 3, 1032, 0.8), (12289, 16, 1032, 0.97), (40007, 2, 264, 0.9),
                                        (20001, 8, 1040, 0.0), (70001, 1, 520, 0.5), (50000, 3, 264, 1.0)])
def test_combine_grad_of_many_tokens(M, k, H, drop):
    """Many tokens with few rows or none: the same bits as in calls on a few of them, whatever the others hold."""
    say("combine_grad of many %s" % ((M, k, H, drop),))
    rng = np.random.default_rng([M, k, H])
    valid = rng.random((M, k)) >= drop
    R = max(int(valid.sum()), 1)
    pos = np.where(valid, 0, rng.choice([-1, R, R + 7, -2 ** 31], size=(M, k))).astype(np.int32)
    pos[valid] = rng.permutation(int(valid.sum()))
    torch.manual_seed(M)
    dy = torch.randn(M, H, device=DEV).to(torch.bfloat16)
    tv = torch.from_numpy(valid).to(DEV)
    dy[~tv.any(1)] = float("nan")
    rows = torch.randn(R, H, device=DEV).to(torch.bfloat16)
    tp, w = torch.from_numpy(pos).to(DEV), torch.randn(M, k, device=DEV)
    canvas = Canvas(R, H, torch.bfloat16)
    drows, dw = moe.combine_grad(dy, rows, tp, w, canvas.t)
    canvas.check_untouched(np.full(R, bool(valid.any())))
    assert not bool(dw[~tv].any())
    ref = torch.zeros(M, k, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(ref)
    for j in range(k):
        at = tv[:, j]
        terms = dy[at].double() * rows[tp[at, j].long()].double()
        ref[at, j], mag[at, j] = terms.sum(1), terms.abs().sum(1)
    check(dw, f64(ref), f64(mag), H, "dweights")
    for t0 in list(range(0, M, M // 3 + 1)) + [M - 1]:
        part = slice(t0, min(t0 + 999, M))
        few = torch.full_like(rows, 7)
        few, dwf = moe.combine_grad(dy[part], rows, tp[part], w[part], few)
        here = tp[part][tv[part]].long()
        assert torch.equal(dwf, dw[part]) and torch.equal(few[here], drows[here])


@pytest.mark.parametrize("M,k,E", [(1, 1, 1), (1, 8, 64), (7, 16, 512), (333, 3, 7), (5000, 8, 128), (64, 2, 65)])
def test_route_grad(M, k, E):
    rng = np.random.default_rng([M, k, E])
    logits = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32) * 3).to(DEV)
    ids, w = moe.route_topk(logits, k)
    d = torch.from_numpy(rng.standard_normal((M, k)).astype(np.float32)).to(DEV)
    got = f64(moe.route_topk_grad(ids, w, d, E))
    wn, dn, at = f64(w), f64(d), ids.cpu().numpy()
    mean = (wn * dn).sum(1, keepdims=True)
    ref = np.zeros((M, E))
    tol = np.zeros((M, E))
    np.put_along_axis(ref, at, wn * (dn - mean), 1)
    # the mean's sum of k terms, the difference and the product
    np.put_along_axis(tol, at, wn * sum_bound(k, np.abs(wn * dn).sum(1, keepdims=True) + np.abs(dn)), 1)
    assert (np.abs(got - ref) <= tol).all()
    # against differences of the softmax itself, in 64 bits
    if M > 64:
        return
    z = f64(logits)
    for m in range(M):
        for e in at[m][:3]:
            h = 1e-5
            f = []
            for s in (h, -h):
                q = z[m].copy()
                q[e] += s
                p = np.exp(q[at[m]] - q[at[m]].max())
                f.append((p / p.sum() * dn[m]).sum())
            # the difference's own error, h^2 times a third derivative of at most sum|d|, and the rounding of its terms
            bound = (1e-9 + tol[m, e] + 2.0 ** -23) * (1 + np.abs(dn[m]).sum())
            assert abs((f[0] - f[1]) / (2 * h) - got[m, e]) <= bound


def test_route_grad_ids_outside_and_equal():
    ids = torch.tensor([[0, -1, 2], [3, 3, 1], [9, 9, 9]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, float("nan"), 0.25], [0.25, 0.5, 0.125], [1.0, 1.0, 1.0]], device=DEV)
    d = torch.tensor([[1.0, float("nan"), 2.0], [1.0, 2.0, 4.0], [1.0, 1.0, 1.0]], device=DEV)
    # exact: every value is a sum of few powers of two
    got = moe.route_topk_grad(ids, w, d, 4).cpu().numpy()
    m0, m1 = 0.5 * 1 + 0.25 * 2, 0.25 + 1.0 + 0.5
    assert got[0].tolist() == [0.5 * (1 - m0), 0, 0.25 * (2 - m0), 0]
    assert got[1].tolist() == [0, 0.125 * (4 - m1), 0, 0.25 * (1 - m1) + 0.5 * (2 - m1)]
    assert not got[2].any()


def test_gradient_is_the_combines_own():
    """combine_grad and dispatch against differences of the functions that they are the gradients of."""
    rng = np.random.default_rng(8)
    M, k, E, H = 6, 3, 5, 16
    ids = torch.from_numpy(routing(rng, M, k, E, drop=0.2)).to(DEV)
    x = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(DEV)
    rows, off, pos, _ = moe.dispatch(x, ids, E)
    rows[int(off[E]):] = 0
    w = torch.from_numpy(rng.random((M, k)).astype(np.float32)).to(DEV)
    dy = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(DEV)
    drows, dw = moe.combine_grad(dy, rows, pos, w, torch.zeros_like(rows))
    dx = moe.combine(drows, pos)

    def loss(x_, w_):
        r = moe.dispatch(x_, ids, E, torch.zeros_like(rows))[0]
        return float((moe.combine(r, pos, w_).double() * dy.double()).sum())

    # the loss is linear in each: a difference is off by its values' rounding only, fp32 sums of a few terms
    scale = float((w[:, :, None].double().abs() * dy[:, None].double().abs()).sum()) * float(x.abs().max())
    for t, g in ((0, dx), (1, dw)):
        args = [x, w]
        base = args[t]
        for _ in range(8):
            d = torch.zeros_like(base)
            i = tuple(int(rng.integers(n)) for n in base.shape)
            d[i] = 1.0
            up, dn = list(args), list(args)
            up[t], dn[t] = base + d, base - d
            assert abs((loss(*up) - loss(*dn)) / 2 - float(g[i])) <= scale * 16 * 2.0 ** -24


def test_training_step():
    """The expert half of a layer with its rows copied: forward and all gradients against the formula in 64 bits."""
    rng = np.random.default_rng(21)
    M, k, E, H, I = 150, 3, 6, 136, 72
    x = bf16(rng, M, H)
    logits = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32))
    logits[:, 2] -= 100.0  # an expert without rows
    w13, w2 = bf16(rng, E, 2 * I, H, scale=H ** -0.5), bf16(rng, E, H, I, scale=I ** -0.5)
    dy = bf16(rng, M, H)
    gx, g13, g2, gdy = (t.to(DEV) for t in (x, w13, w2, dy))
    ids, w = moe.route_topk(logits.to(DEV), k)
    rows, off, pos, pairs = moe.dispatch(gx, ids, E)
    gu = moe.grouped_gemm(rows, g13, off)
    h, codes, scales = moe.swiglu_checkpoint(gu, num_rows=off[E:])
    o = moe.grouped_gemm(h, g2, off)
    y = moe.combine(o, pos, w)
    do, dw = moe.combine_grad(gdy, o, pos, w)
    dlogits = moe.route_topk_grad(ids, w, dw, E)
    dh = moe.grouped_gemm_dgrad(do, g2, off)
    dgu, h2, _ = moe.swiglu_checkpoint_grad(codes, scales, dh, num_rows=off[E:])
    dw2 = moe.grouped_gemm_wgrad(do, h2, off)
    dw13 = moe.grouped_gemm_wgrad(dgu, rows, off)
    dx = moe.combine(moe.grouped_gemm_dgrad(dgu, g13, off), pos)
    torch.cuda.synchronize()

    ref = [t.to(torch.float64).requires_grad_() for t in (x, logits, w13, w2)]
    rx, rl, r13, r2 = ref
    rid = ids.cpu().long()
    rw = torch.softmax(torch.gather(rl, 1, rid), 1)
    out = torch.zeros(M, H, dtype=torch.float64)
    for e in range(E):
        t, j = torch.where(rid == e)
        g, u = (rx[t] @ r13[e].T).split(I, 1)
        out = out.index_add(0, t, rw[t, j, None] * ((torch.nn.functional.silu(g) * u) @ r2[e].T))
    (out * dy.to(torch.float64)).sum().backward()

    def close(got, want, bound):
        d = f64(got) - want.detach().numpy()
        assert np.linalg.norm(d) <= bound * np.linalg.norm(want.detach().numpy())

    # roundings to bf16 are at most 2^-8 of each value (about 2^-9.8 of it on average), to e4m3 at most 2^-4 (2^-5.8):
    # y passes three of the former in a row; dlogits the same and dw's sum of rounded terms; the others also the
    # checkpoint's, twice in a product (g and u), which is 2 * 2^-4 of each value at most
    close(y, out, 4 * BF16_STEP)
    close(dlogits, rl.grad, 6 * BF16_STEP)
    for got, want in ((dx, rx), (dw13, r13), (dw2, r2)):
        close(got, want.grad, 2 * 2.0 ** -4 + 6 * BF16_STEP)
    assert not bool(dw2[2].any()) and not bool(dw13[2].any())
