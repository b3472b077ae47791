"""Expert products in 8-bit integers on the GPU: the codes against the rational
definition, the products against exact integer sums; ragged and empty experts,
odd sizes, strides, gathered and scattered rows, padding ids, rows that nothing
may read, few rows (the streamed form) and many (the tiled one); and a layer of
them together."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import BF16_STEP, DEV, Canvas, bf16, f64, offsets_of, poisoned

pytestmark = pytest.mark.gpu

COUNTS = {
    "one_row": [1],
    "two_of_three": [3, 0, 2],
    "decode": [1, 0, 0, 2, 0, 1, 0, 0, 0, 3, 1, 0, 0, 1, 0, 0, 18, 0, 0, 1],
    "few": [9, 16, 17, 0, 31, 32, 33, 8, 1, 0],
    "edges_64": [63, 64, 65, 0, 1],
    "edges_128": [127, 128, 129],
    "edges_256": [255, 0, 256, 257],
    "skewed": [700, 1, 0, 5, 33, 90, 0],
}
SIZES = [(8, 16), (16, 80), (136, 64), (264, 208), (256, 256), (520, 400)]
EXTRA = 5  # rows behind the last expert


def int8_of(x):
    """(codes, scales in 64 bits) of float64 rows, by the definition: 127 x / top is a tie or far from one."""
    top = np.abs(x).max(axis=1, keepdims=True)
    safe = np.where(top > 0, top, 1.0)
    return np.rint(127.0 * x / safe), np.where(top > 0, top / 127.0, 1.0)[:, 0]


def check_codes(codes, scales, x):
    q, s = int8_of(x)
    assert np.array_equal(codes.cpu().numpy().astype(np.float64), q)
    # one rounding to fp32, which below its normal range is an absolute one
    assert (np.abs(f64(scales) - s) <= 2.0 ** -24 * s + 2.0 ** -149).all()


@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (9, 1008), (5, 1024), (4, 1040), (6, 2048), (7, 2064), (3, 4096),
                                 (5, 4112), (2, 8208), (3, 16384), (2, 16400), (1, 40000), (2, 65536), (4000, 64)])
def test_quant(M, K):
    say("quant M=%d K=%d" % (M, K))
    rng = np.random.default_rng([M, K])
    x = bf16(rng, M, K, scale=2.0) * torch.from_numpy(np.exp(rng.standard_normal((M, 1)))).to(torch.bfloat16)
    guard = torch.full((M * K + 64,), 99, dtype=torch.int8, device=DEV)
    codes = guard[32:32 + M * K].view(M, K)
    got, scales = moe.quant_int8(poisoned(x, 8), codes)
    torch.cuda.synchronize()
    assert got.data_ptr() == codes.data_ptr()
    assert bool((guard[:32] == 99).all()) and bool((guard[-32:] == 99).all())
    check_codes(got, scales, f64(x))


def test_quant_every_quotient():
    # every pair of 8-bit mantissas: all ties there can be between two codes, and all quotients next to one
    m = np.arange(128, 256)
    rows = []
    for e in range(0, 9):
        rows += [np.concatenate([[t], m * 2.0 ** -e * np.where(m * 2.0 ** -e <= t, 1, 0.5)]) for t in m]
    x = np.zeros((len(rows), 144))
    x[:, :129] = np.array(rows)
    x[:, 1:] *= np.where(np.arange(143) % 2, -1.0, 1.0)
    t = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(f64(t), x)
    for shift in (1.0, 2.0 ** -120, 2.0 ** 110):
        codes, scales = moe.quant_int8((t * shift).to(DEV))
        check_codes(codes, scales, x * shift)


def test_quant_special_rows():
    x = torch.zeros(6, 32, dtype=torch.bfloat16)
    x[1, 3] = float("inf")
    x[2, 4], x[2, 5] = float("nan"), 7.0
    x[3, 31] = -3.0
    x[4, :3] = torch.tensor([2.0 ** -133, -2.0 ** -132, 2.0 ** -126])  # the smallest of the type
    x[5, :2] = torch.tensor([torch.finfo(torch.bfloat16).max, -2.0 ** 120])
    codes, scales = moe.quant_int8(x.to(DEV))
    c, s = codes.cpu(), scales.cpu()
    assert not bool(c[:3].any()) and s[0] == 1.0 and bool(torch.isnan(s[1:3]).all())
    check_codes(codes[3:], scales[3:], f64(x[3:]))


@pytest.mark.parametrize("R,I", [(1, 16), (5, 144), (9, 768), (3, 1040), (6, 2048), (2, 4096), (3, 7184), (2, 14336),
                                 (2, 20000), (1, 65536)])
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu(R, I, weighted):
    say("swiglu_int8 R=%d I=%d %s" % (R, I, weighted))
    rng = np.random.default_rng([R, I])
    gu = bf16(rng, R + 2, 2 * I, scale=2.0)
    gu[R:] = float("nan")
    w = rng.random(R + 2).astype(np.float32) - 0.3
    codes = torch.full((R + 2, I), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((R + 2,), -7.75, device=DEV)
    moe.swiglu_int8(poisoned(gu, 8), torch.from_numpy(w).to(DEV) if weighted else None,
                    num_rows=torch.tensor([R], dtype=torch.int32, device=DEV), codes=codes, scales=scales)
    torch.cuda.synchronize()
    assert bool((codes[R:] == 99).all()) and bool((scales[R:] == -7.75).all())
    g, u = f64(gu)[:R, :I], f64(gu)[:R, I:]
    h = g / (1 + np.exp(-g)) * u
    top = np.abs(h).max(axis=1, keepdims=True)
    # h in fp32: the exponent's argument is off by 2^-24 of its size (at most |g| * 1.45), exp2, reciprocal and four
    # products by an ulp each, so h by (1.45 |g| + 8) * 2^-23 of its size, and the row's largest likewise
    rel = (1.45 * np.abs(g).max() + 8) * 2.0 ** -23
    assert rel < 1e-5
    assert (np.abs(127.0 * h / top - codes[:R].cpu().numpy()) <= 0.5 + 127 * 2 * rel).all()
    s = top[:, 0] / 127.0 * (w[:R].astype(np.float64) if weighted else 1.0)
    assert (np.abs(f64(scales[:R]) - s) <= (rel + 2.0 ** -23) * np.abs(s)).all()


def test_swiglu_special_rows():
    gu = torch.zeros(5, 64, dtype=torch.bfloat16)
    gu[1, 3], gu[1, 35] = float("inf"), 1.0
    gu[2, 3] = float("nan")
    gu[3, :32], gu[3, 32:] = -300.0, 1.0  # the activation's exponential overflows: zeros
    gu[4, 0], gu[4, 32] = 200.0, -2.0
    codes, scales = moe.swiglu_int8(gu.to(DEV))
    s = scales.cpu()
    assert s[0] == 1.0 and bool(torch.isnan(s[1:3]).all()) and s[3] == 1.0
    assert not bool(codes[:4].any()) and codes[4, 0] == -127 and abs(float(s[4]) - 400.0 / 127) < 1e-5


def rows_operand(rng, R, K, gather, div, pad):
    """(codes view, scales, ids or None, grouped codes, grouped scales): what no row may read has NaN scales."""
    n = R if not gather else max(2, R // div + 2)
    codes = rng.integers(-128, 128, (n, K), dtype=np.int8)
    scales = np.exp(rng.standard_normal(n)).astype(np.float32)
    full = torch.full((n, K + pad), 77, dtype=torch.int8, device=DEV)
    full[:, :K] = torch.from_numpy(codes).to(DEV)
    if not gather:
        scales[R - EXTRA:] = np.nan
        return full[:, :K], scales, None, codes, scales
    scales[n - 1] = np.nan
    ids = rng.integers(0, (n - 1) * div, R).astype(np.int32)
    ids[rng.random(R) < 0.1] = n * div  # padding ids: zeros
    ids[R - EXTRA:] = (n - 1) * div
    ids[:1] = -1 if R > 4 + EXTRA else ids[:1]
    ok = (ids >= 0) & (ids // div < n)
    at = np.where(ok, ids // div, 0)
    return full[:, :K], scales, ids, codes[at] * ok[:, None].astype(np.int8), np.where(ok, scales[at], 0.0)


def run_product(counts, N, K, gather, scatter, dtype, seed=0, div=3):
    say("int8 %s N=%d K=%d gather=%s scatter=%s %s" % (counts[:12], N, K, gather, scatter, dtype))
    rng = np.random.default_rng([seed, N, K, len(counts)])
    E, off, R = len(counts), offsets_of(counts), int(sum(counts)) + EXTRA
    w = rng.integers(-128, 128, (E, N, K), dtype=np.int8)
    ws = (np.exp(rng.standard_normal((E, N))) * 0.01).astype(np.float32)
    ws[np.array(counts) == 0] = np.nan  # an expert without rows is not read into any result
    a, s, ids, rows, rs = rows_operand(rng, R, K, gather, div, 16)
    total = off[-1]
    canvas = Canvas(R + 4 if scatter else R, N, dtype)
    place, to = np.arange(R, dtype=np.int32), None
    if scatter:
        place = rng.permutation(R + 4)[:R].astype(np.int32)
        place[::11] = -1
        place[3::13] = R + 4
        to = torch.from_numpy(place).to(DEV)
    place = place[:total]
    got = moe.grouped_gemm_int8(a, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV),
                                torch.from_numpy(off).to(DEV), canvas.t, a_scale=torch.from_numpy(s).to(DEV),
                                a_rows=None if ids is None else torch.from_numpy(ids).to(DEV),
                                a_div=div if gather else 1, out_rows=to)
    torch.cuda.synchronize()
    assert got.data_ptr() == canvas.t.data_ptr()
    keep = (place >= 0) & (place < canvas.t.shape[0])
    written = np.zeros(canvas.t.shape[0], dtype=bool)
    written[place[keep]] = True
    canvas.check_untouched(written)
    ref = np.zeros((total, N))
    for e in range(E):
        sl = slice(off[e], off[e + 1])
        if counts[e]:
            ref[sl] = rows[sl].astype(np.float64) @ w[e].T.astype(np.float64)
            ref[sl] *= rs[sl, None].astype(np.float64) * ws[e].astype(np.float64)
    g, ref = f64(canvas.t)[place[keep]], ref[keep]
    # the exact sum's conversion and two products, rounded to fp32 each; then the type
    tol = 3.01 * 2.0 ** -24 + (1.01 * BF16_STEP if dtype == torch.bfloat16 else 0.0)
    bad = ~(np.abs(g - ref) <= tol * np.abs(ref))
    assert not bad.any(), "%d of %d off, first at %s: %r for %r" % (bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0],
                                                                     ref[bad][0])


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", SIZES)
def test_product(name, N, K):
    run_product(COUNTS[name], N, K, False, False, torch.bfloat16)


@pytest.mark.parametrize("gather,scatter", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["two_of_three", "decode", "few", "edges_64", "edges_256", "skewed"])
def test_product_rows(gather, scatter, dtype, name):
    run_product(COUNTS[name], 264, 336, gather, scatter, dtype)


@pytest.mark.parametrize("name", ["one_row", "decode", "few", "edges_64"])
@pytest.mark.parametrize("K", [16, 128, 144, 384, 512, 640, 656, 1024, 1040, 1168, 2064, 4112])
@pytest.mark.parametrize("N,dtype", [(2056, torch.float32), (8200, torch.bfloat16)])
def test_product_steps(name, K, N, dtype):
    # every number of steps that a wave or the four share, and parts of one; bands of each width
    run_product(COUNTS[name], N, K if N < 8200 else min(K, 1040), True, True, dtype)


@pytest.mark.parametrize("counts,N", [([700, 640, 0, 720, 1, 129, 900], 8200),
                                      ([64 * (i % 3) + 33 for i in range(90)], 1544)])
@pytest.mark.parametrize("K", [16, 80, 208, 656])
@pytest.mark.parametrize("gather,scatter,dtype", [(False, False, torch.bfloat16), (True, False, torch.float32),
                                                  (True, True, torch.bfloat16), (False, True, torch.float32)])
def test_tiles(counts, N, K, gather, scatter, dtype):
    # results whose tiles fill the GPU: the tiled form
    run_product(counts, N, K, gather, scatter, dtype)


@pytest.mark.parametrize("name", ["edges_64", "edges_128", "edges_256", "skewed"])
@pytest.mark.parametrize("K,dtype", [(656, torch.bfloat16), (784, torch.float32)])
def test_tile_edges(name, K, dtype):
    run_product(COUNTS[name], 8200, K, name == "skewed", name == "edges_128", dtype)


@pytest.mark.parametrize("counts", [[300], [64, 65, 0, 129], [1000, 1]])
@pytest.mark.parametrize("N,K", [(24, 144), (184, 3888), (520, 272)])
def test_passes_side_by_side(counts, N, K):
    # narrow results of many rows: the passes of a band on workgroups of their own
    run_product(counts, N, K, True, True, torch.bfloat16)
    run_product(counts, N, K, False, False, torch.float32)


MANY = {  # several tiles of each kind for every workgroup
    "whole": [2100, 700, 0, 2900, 1500],
    "halves": [70 + i % 59 for i in range(40)],
    "small": [1 + i % 64 for i in range(48)],
    "mixed": [256 * (i % 3) + (37 * i) % 256 for i in range(30)],
}


@pytest.mark.parametrize("name", list(MANY))
@pytest.mark.parametrize("K", [144, 400, 656])
def test_many_tiles_per_workgroup(name, K):
    run_product(MANY[name], 4360, K, K == 400, K == 656, torch.bfloat16)


@pytest.mark.parametrize("name,K", [("two_of_three", 65536), ("edges_64", 131056)])
def test_largest_sums(name, K):
    # -128 times -128 throughout: the largest sums there are, below 2^31
    counts = COUNTS[name]
    off, R = offsets_of(counts), int(sum(counts))
    a = torch.full((R, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((len(counts), 8, K), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(len(counts), 8, device=DEV)
    y = moe.grouped_gemm_int8(a, w, one, torch.from_numpy(off).to(DEV), a_scale=torch.ones(R, device=DEV),
                              out_dtype=torch.float32)
    assert bool((y == float(16384 * K)).all())


@pytest.mark.parametrize("name", ["one_row", "decode", "few", "skewed"])
@pytest.mark.parametrize("gather", [False, True])
def test_product_of_bf16_rows(name, gather):
    """bf16 rows are quantised by the call: the same bits as in two steps."""
    rng = np.random.default_rng(17)
    counts, N, K, div = COUNTS[name], 136, 272, 3
    off, R = offsets_of(counts), int(sum(counts))
    n = R if not gather else R // div + 1
    a = bf16(rng, n, K)
    a[n - 1, 3] = float("nan")  # its scale, and with it its results
    a[n // 2] = 0.0
    a = poisoned(a, 8)
    ids = torch.from_numpy(rng.integers(-1, n * div + 2, R).astype(np.int32)).to(DEV) if gather else None
    w, ws = moe.quant_int8(bf16(rng, len(counts) * N, K).to(DEV))
    w, ws = w.view(-1, N, K), ws.view(-1, N)
    g_off = torch.from_numpy(off).to(DEV)
    kw = dict(a_rows=ids, a_div=div if gather else 1)
    one = moe.grouped_gemm_int8(a, w, ws, g_off, **kw)
    codes, s = moe.quant_int8(a)
    two = moe.grouped_gemm_int8(codes, w, ws, g_off, a_scale=s, **kw)
    assert torch.equal(one.view(torch.int16), two.view(torch.int16))


@pytest.mark.parametrize("counts", [[1] * 16, [2, 0, 0, 5, 1, 0, 0, 0], [0] * 9 + [17], [0] * 11 + [33, 1]])
@pytest.mark.parametrize("N,K", [(8, 16), (200, 1168), (2056, 2064), (1032, 6160)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_on_the_way(counts, N, K, dtype):
    """Few bf16 rows, whose codes are made inside the product: the same bits as in two steps."""
    say("codes on the way %s N=%d K=%d" % (counts, N, K))
    rng = np.random.default_rng([len(counts), N, K])
    off, R = offsets_of(counts), int(sum(counts))
    a = poisoned(bf16(rng, R, K) * torch.from_numpy(np.exp(rng.standard_normal((R, 1)))).to(torch.bfloat16), 8)
    w = torch.from_numpy(rng.integers(-128, 128, (len(counts), N, K), dtype=np.int8)).to(DEV)
    ws = torch.rand(len(counts), N, device=DEV)
    g_off = torch.from_numpy(off).to(DEV)
    assert moe.load().moe_grouped_int8_workspace_size(R, len(counts), N, K, R) == 0
    one = moe.grouped_gemm_int8(a, w, ws, g_off, out_dtype=dtype)
    codes, s = moe.quant_int8(a)
    assert torch.equal(one, moe.grouped_gemm_int8(codes, w, ws, g_off, a_scale=s, out_dtype=dtype))


def test_no_rows():
    w = torch.zeros(3, 16, 32, dtype=torch.int8, device=DEV)
    ws, off = torch.ones(3, 16, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    for a, s in ((torch.empty(0, 32, dtype=torch.bfloat16, device=DEV), None),
                 (torch.empty(0, 32, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV))):
        assert moe.grouped_gemm_int8(a, w, ws, off, a_scale=s).shape == (0, 16)
    assert [t.shape for t in moe.quant_int8(torch.empty(0, 32, dtype=torch.bfloat16, device=DEV))] == [(0, 32), (0,)]
    assert [t.shape for t in moe.swiglu_int8(torch.empty(0, 32, dtype=torch.bfloat16, device=DEV))] == [(0, 16), (0,)]
    # rows without experts: nothing is written
    out = torch.full((4, 16), -7.75, device=DEV)
    moe.grouped_gemm_int8(torch.ones(4, 32, dtype=torch.bfloat16, device=DEV), w, ws, off, out)
    assert bool((out == -7.75).all())


def test_nan_row_stays_its_own():
    rng = np.random.default_rng(2)
    counts = [40, 3, 30]
    x = bf16(rng, 73, 64)
    x[41, 7] = float("inf")
    w, ws = moe.quant_int8(bf16(rng, 3 * 24, 64).to(DEV))
    ok = torch.isfinite(moe.grouped_gemm_int8(x.to(DEV), w.view(3, 24, 64), ws.view(3, 24),
                                              torch.from_numpy(offsets_of(counts)).to(DEV)))
    assert not bool(ok[41].any()) and bool(ok[:41].all()) and bool(ok[42:].all())


@pytest.mark.parametrize("M,k,E", [(1, 2, 8), (33, 4, 16), (400, 3, 6)])
def test_layer(M, k, E):
    """A layer in 8-bit integers: the tokens' products, the activation, the down products and the combine, against
    the same of the values that the codes stand for."""
    rng = np.random.default_rng([M, k, E])
    H, I = 256, 144
    x = bf16(rng, M, H)
    logits = torch.from_numpy(rng.standard_normal((M, E)).astype(np.float32)).to(DEV)
    w13, s13 = moe.quant_int8(bf16(rng, E * 2 * I, H, scale=H ** -0.5).to(DEV))
    w2, s2 = moe.quant_int8(bf16(rng, E * H, I, scale=I ** -0.5).to(DEV))
    ids, w = moe.route_topk(logits, k)
    _, off, pos, pairs = moe.dispatch(None, ids, E)
    gu = moe.grouped_gemm_int8(x.to(DEV), w13.view(E, 2 * I, H), s13.view(E, 2 * I), off, a_rows=pairs, a_div=k)
    codes, scales = moe.swiglu_int8(gu, num_rows=off[E:])
    o = moe.grouped_gemm_int8(codes, w2.view(E, H, I), s2.view(E, H), off, a_scale=scales)
    y = moe.combine(o, pos, w)
    # weighted in the activation's scales, and back in pair order
    codes, scales = moe.swiglu_int8(gu, w.view(-1)[pairs.long()])
    o = moe.grouped_gemm_int8(codes, w2.view(E, H, I), s2.view(E, H), off, a_scale=scales, out_rows=pairs)
    y2 = moe.combine(o, torch.arange(M * k, dtype=torch.int32, device=DEV).view(M, k))
    torch.cuda.synchronize()
    q, s = int8_of(f64(x))
    v13, v2 = (f64(c).reshape(E, -1, n) * f64(t).reshape(E, -1, 1) for c, t, n in ((w13, s13, H), (w2, s2, I)))
    ref, mag = np.zeros((M, H)), np.zeros((M, H))
    for t in range(M):
        for j, e in enumerate(ids[t].tolist()):
            g, u = np.split(v13[e] @ (q[t] * s[t]), 2)
            h = g / (1 + np.exp(-g)) * u
            # gu is rounded to bf16, which h feels twice (the gate's slope is at most 1.1 |SiLU| + 1 of its change);
            # then half a code of the row's largest; o is rounded to bf16
            slack = BF16_STEP * (np.abs(h) * 1.1 + (1.1 * np.abs(g) + 1e-3) * np.abs(u) * 1.1) + np.abs(h).max() / 254
            wt = float(w[t, j])
            ref[t] += wt * (v2[e] @ h)
            mag[t] += wt * (np.abs(v2[e]) @ slack + BF16_STEP * (np.abs(v2[e]) @ np.abs(h)))
    for got in (y, y2):
        assert (np.abs(f64(got) - ref) <= 1.02 * mag + BF16_STEP * np.abs(ref)).all()
