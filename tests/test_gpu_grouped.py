"""Grouped expert products and their gradients on the GPU against plain sums
in 64 bits: ragged and empty experts, odd sizes, strides, gathered and
scattered rows, padding ids, rows behind the last expert, NaN next to what a
result may read."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV, Canvas, bf16, check, f64, offsets_of, poisoned, w4_values

pytestmark = pytest.mark.gpu

COUNTS = {
    "one_row": [1],
    "two_of_three": [3, 0, 2],
    "edges_64": [63, 64, 65, 0, 1],
    "edges_128": [127, 128, 129],
    "edges_256": [255, 0, 256, 257],
    "skewed": [700, 1, 0, 5, 33, 90, 0],
    "many_small": [1, 2, 0, 3, 1, 0, 7, 4, 2, 1, 0, 0, 5, 1, 9, 17, 16, 15, 31, 32],
}
SIZES = [(8, 8), (16, 72), (136, 64), (264, 200), (256, 256), (520, 392)]
EXTRA = 5  # rows behind the last expert


def operands(rng, counts, width, gather, div=3, pad=8):
    """A rows operand of `width` for the counts: (GPU tensor, ids or None, its
    grouped rows float64).  Everything no row may read holds NaN."""
    R = int(sum(counts)) + EXTRA
    if not gather:
        t = bf16(rng, R, width)
        t[R - EXTRA:] = float("nan")
        return poisoned(t, pad), None, f64(t)
    M = max(1, R // div + 2)
    t = bf16(rng, M, width)
    ids = rng.integers(0, (M - 1) * div, R).astype(np.int32)
    t[M - 1] = float("nan")  # no id reaches the last row
    ids[rng.random(R) < 0.1] = M * div  # padding ids: zeros
    ids[R - EXTRA:] = (M - 1) * div  # rows that belong to no expert
    ids[:1] = -1 if R > 4 else ids[:1]
    rows = np.zeros((R, width))
    ok = (ids >= 0) & (ids // div < M)
    rows[ok] = f64(t)[ids[ok] // div]
    return poisoned(t, pad), torch.from_numpy(ids).to(DEV), rows


def reference(kind, rows, w, off):
    """(result, sum of absolute terms) of the grouped rows, float64."""
    E, N, K = w.shape
    out = np.zeros((rows.shape[0], K if kind == "dgrad" else N))
    mag = np.zeros_like(out)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        m = w[e] if kind == "dgrad" else w[e].T
        out[s], mag[s] = rows[s] @ m, np.abs(rows[s]) @ np.abs(m)
    return out, mag


def product(kind, a, w, off, **kw):
    if kind == "dgrad":
        return moe.grouped_gemm_dgrad(a, w, off, kw["out"], dy_rows=kw["ids"], dy_div=kw["div"],
                                      out_rows=kw["out_rows"])
    return moe.grouped_gemm(a, w, off, kw["out"], a_rows=kw["ids"], a_div=kw["div"], out_rows=kw["out_rows"])


def run_product(kind, name, N, K, gather, scatter, dtype, seed=0):
    counts = COUNTS[name]
    say("%s %s N=%d K=%d gather=%s scatter=%s %s" % (kind, name, N, K, gather, scatter, dtype))
    rng = np.random.default_rng([seed, N, K, len(counts)])
    E, off = len(counts), offsets_of(counts)
    src, dst = (N, K) if kind == "dgrad" else (K, N)
    w = bf16(rng, E, N, K, scale=src ** -0.5)
    for e in range(E):
        if counts[e] == 0:
            w[e] = float("nan")  # an expert without rows is not read into any result
    a, ids, rows = operands(rng, counts, src, gather)
    R = rows.shape[0]
    wz = np.where(np.isnan(f64(w)), 0.0, f64(w))
    ref, mag = reference(kind, rows, wz, off)
    total = off[-1]
    to = None
    canvas = Canvas(R + 4 if scatter else R, dst, dtype)
    place = np.arange(total)
    if scatter:
        place = rng.permutation(R + 4)[:R].astype(np.int32)
        place[::11] = -1
        place[3::13] = R + 4
        to = torch.from_numpy(place).to(DEV)
        place = place[:total]
    got = product(kind, a, w.to(DEV), torch.from_numpy(off).to(DEV), out=canvas.t, ids=ids, div=3, out_rows=to)
    torch.cuda.synchronize()
    assert got.data_ptr() == canvas.t.data_ptr()
    keep = (place >= 0) & (place < canvas.t.shape[0])
    written = np.zeros(canvas.t.shape[0], dtype=bool)
    written[place[keep]] = True
    canvas.check_untouched(written)
    check(canvas.t[torch.from_numpy(place[keep].astype(np.int64)).to(DEV)], ref[:total][keep], mag[:total][keep], src,
          "%s %s" % (kind, name))


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", SIZES)
def test_product(kind, name, N, K):
    run_product(kind, name, N, K, False, False, torch.bfloat16)


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("gather,scatter", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["two_of_three", "edges_64", "edges_256", "skewed", "many_small"])
def test_product_rows(kind, gather, scatter, dtype, name):
    run_product(kind, name, 264, 328, gather, scatter, dtype)


MANY = {  # several tiles of each kind for every workgroup
    "whole": [2100, 700, 0, 2900, 1500],
    "halves": [70 + i % 59 for i in range(40)],
    "small": [1 + i % 64 for i in range(48)],
    "mixed": [256 * (i % 3) + (37 * i) % 256 for i in range(30)],
}


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("name", list(MANY))
@pytest.mark.parametrize("inner", [72, 200, 328])
def test_many_tiles_per_workgroup(kind, name, inner, monkeypatch):
    monkeypatch.setitem(COUNTS, name, MANY[name])
    N, K = (4360, inner) if kind == "fwd" else (inner, 4360)
    run_product(kind, name, N, K, inner == 200, inner == 328, torch.bfloat16)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)])
@pytest.mark.parametrize("counts", [[130, 1, 0, 64, 300, 65, 129, 128], [5] * 12])
def test_wgrad_many_tiles_per_workgroup(gather, dtype, accumulate, counts, monkeypatch):
    monkeypatch.setitem(COUNTS, "many", counts)
    wgrad_case("many", 4360, 1544, False, gather, dtype, accumulate)


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
def test_long_contraction(kind):
    # the contraction runs over 4104 terms, one 64-step and 8 more past 64 whole ones
    N, K = (136, 4104) if kind == "fwd" else (4104, 136)
    run_product(kind, "edges_64", N, K, False, False, torch.float32)


def wgrad_case(name, N, K, gather_dy, gather_a, dtype, accumulate=False):
    counts = COUNTS[name]
    say("wgrad %s N=%d K=%d gather=%s,%s %s acc=%s" % (name, N, K, gather_dy, gather_a, dtype, accumulate))
    rng = np.random.default_rng([7, N, K, len(counts)])
    off = offsets_of(counts)
    dy, idy, rdy = operands(rng, counts, N, gather_dy)
    a, ida, ra = operands(rng, counts, K, gather_a, div=2)
    E = len(counts)
    start = torch.from_numpy(rng.standard_normal((E, N, K)).astype(np.float32))
    guard = torch.full((E * N * K + 128,), -7.75, dtype=dtype, device=DEV)
    out = guard[64:64 + E * N * K].view(E, N, K)
    if accumulate:
        out.copy_(start)
    got = moe.grouped_gemm_wgrad(dy, a, torch.from_numpy(off).to(DEV), out, dy_rows=idy, dy_div=3, a_rows=ida, a_div=2,
                                 accumulate=accumulate)
    torch.cuda.synchronize()
    assert bool((guard[:64] == -7.75).all()) and bool((guard[-64:] == -7.75).all())
    for e in range(E):
        x, y = rdy[off[e]:off[e + 1]], ra[off[e]:off[e + 1]]
        ref, mag = x.T @ y, np.abs(x).T @ np.abs(y)
        if accumulate:
            s = f64(start[e])
            # one more fp32 addition
            check(got[e], ref + s, mag + np.abs(s), counts[e] + 1, "expert %d" % e)
            if counts[e] == 0:
                assert torch.equal(got[e].cpu(), start[e])
        else:
            check(got[e], ref, mag, counts[e], "expert %d" % e)
            if counts[e] == 0:
                assert not bool(got[e].any())


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", SIZES)
def test_wgrad(name, N, K):
    wgrad_case(name, N, K, False, False, torch.float32)


@pytest.mark.parametrize("gather_dy,gather_a", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)])
@pytest.mark.parametrize("name", ["two_of_three", "edges_64", "edges_256", "skewed"])
def test_wgrad_rows(gather_dy, gather_a, dtype, accumulate, name):
    wgrad_case(name, 264, 328, gather_dy, gather_a, dtype, accumulate)


def test_nan_stays_with_its_expert():
    rng = np.random.default_rng(3)
    counts = [70, 50, 130]
    off = torch.from_numpy(offsets_of(counts)).to(DEV)
    dy, a = bf16(rng, 250, 136), bf16(rng, 250, 200)
    dy[75] = float("nan")
    a[80] = float("inf")
    w = bf16(rng, 3, 136, 200)
    w[1, 5] = float("nan")
    dw = moe.grouped_gemm_wgrad(dy.to(DEV), a.to(DEV), off)
    y = moe.grouped_gemm(a.to(DEV), w.to(DEV), off)
    torch.cuda.synchronize()
    fin = torch.isfinite(dw).flatten(1).all(1).tolist()
    assert fin == [True, False, True]
    ok = torch.isfinite(y)
    assert bool(ok[:70].all()) and bool(ok[120:].all())
    assert not bool(ok[70:120, 5].any()) and not bool(ok[80].any())
    rest = ok[70:120].clone()
    rest[:, 5] = True
    rest[10] = True
    assert bool(rest.all())


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", [(8, 128), (72, 256), (200, 384), (136, 1152), (32, 2176)])
def test_w4(fmt, name, N, K):
    w4_case(fmt, name, N, K, name != "one_row", name == "skewed", torch.float32 if N == 72 else torch.bfloat16)


@pytest.mark.parametrize("K", [32, 96, 160, 1120])
@pytest.mark.parametrize("name", ["one_row", "many_small", "edges_64"])
def test_mxfp4_short_groups(K, name):
    w4_case("mxfp4", name, 72, K, False, False, torch.float32)


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
@pytest.mark.parametrize("name,N,K", [("many_small", 1544, 1408), ("many_small", 2056, 1280), ("many_small", 3400, 640),
                                      ("edges_64", 3400, 1408), ("edges_64", 3400, 640), ("one_row", 16648, 1152),
                                      ("two_of_three", 8328, 384)])
def test_w4_larger(fmt, name, N, K):
    # the launch's wider bands, with K long and short, few and many rows per expert
    w4_case(fmt, name, N, K, True, True, torch.bfloat16)


def w4_case(fmt, name, N, K, gather, scatter, dtype):
    counts = COUNTS[name]
    say("w4 %s %s N=%d K=%d gather=%s scatter=%s %s" % (fmt, name, N, K, gather, scatter, dtype))
    rng = np.random.default_rng([11, N, K, len(counts)])
    E, off = len(counts), offsets_of(counts)
    codes = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = torch.from_numpy(rng.integers(110, 135, (E, N, K // 32), dtype=np.uint8))
    else:
        scales = torch.from_numpy(rng.uniform(0.001, 0.1, (E, N, K // 128)).astype(np.float32)).to(torch.bfloat16)
        scales[:, ::3] *= -1
    a, ids, rows = operands(rng, counts, K, gather)
    w = w4_values(codes, scales, fmt)
    ref, mag = reference("fwd", rows, w, off)
    n = K
    if fmt == "int4":
        # q - 8 may be formed as (16 + q) - 24 inside the sum of a group of 128: terms up to 31 + 24 times |s x|
        mag, n = reference("fwd", np.abs(rows), np.repeat(np.abs(f64(scales)), 128, axis=2) * 55, off)[0], 128 + K // 128
    total = off[-1]
    R = rows.shape[0]
    canvas = Canvas(R, N, dtype)
    place = rng.permutation(R).astype(np.int32) if scatter else np.arange(R, dtype=np.int32)
    to = torch.from_numpy(place).to(DEV) if scatter else None
    moe.grouped_gemm_w4(a, torch.from_numpy(codes).to(DEV), scales.to(DEV), torch.from_numpy(off).to(DEV), canvas.t,
                        a_rows=ids, a_div=3, out_rows=to)
    torch.cuda.synchronize()
    written = np.zeros(R, dtype=bool)
    written[place[:total]] = True
    canvas.check_untouched(written)
    check(canvas.t[torch.from_numpy(place[:total].astype(np.int64)).to(DEV)], ref[:total], mag[:total], n, name)


@pytest.mark.parametrize("fmt,K", [("mxfp4", 6016), ("mxfp4", 6208), ("int4", 6016), ("int4", 6272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_w4_long(fmt, K, dtype):
    # K split over all four waves of a wide band
    w4_case(fmt, "many_small", 1544, K, True, False, dtype)


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
@pytest.mark.parametrize("K", [128, 256, 512, 768, 1024, 1280])
@pytest.mark.parametrize("name", ["many_small", "edges_64"])
def test_w4_steps(fmt, K, name):
    # every number of steps from one to five, and a part of one
    w4_case(fmt, name, 2056, K, False, True, torch.bfloat16)


NARROW = {"one": [1], "full": [64], "first_of_many": [0] * 5 + [1] + [0] * 506, "some": [3, 0, 17, 1, 0, 33, 5],
          "last": [0, 0, 0, 2]}


@pytest.mark.parametrize("name", list(NARROW))
@pytest.mark.parametrize("N,K", [(8, 8), (72, 64), (136, 200), (264, 520), (200, 1088)])
@pytest.mark.parametrize("dtype,scatter", [(torch.bfloat16, False), (torch.float32, True)])
def test_product_few_rows(name, N, K, dtype, scatter, monkeypatch):
    # narrow results of at most 64 rows, with the bound on the rows as small as it may be
    monkeypatch.setitem(COUNTS, name, NARROW[name])
    monkeypatch.setitem(globals(), "EXTRA", 0)
    run_product("fwd", name, N, K, scatter, scatter, dtype)
