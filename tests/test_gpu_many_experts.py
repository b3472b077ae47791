"""Grouped products of more experts than a wave has lanes, of fewer rows than
experts, and with offsets that no routing makes, each on the kernel that serves
it: the tile kernel's prefix sums over up to 512 experts, the weight gradient's
zeros of experts without rows, and the 4-bit products' search for the experts
that hold rows."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
import test_gpu_grouped as grouped
from gpu_common import say
from grouped_common import DEV, Canvas, bf16, check, f64, offsets_of, w4_values

pytestmark = pytest.mark.gpu


def counts_of(E):
    """Mostly empty experts; whole, half and small tiles on both sides of every
    64th expert and at the end."""
    c = [0] * E
    for i in range(0, E, 7):
        c[i] = 1 + i % 5
    for at, n in ((1, 300), (62, 65), (63, 128), (64, 129), (E - 1, 257), (E - 2, 64), (127, 66), (128, 1), (255, 200),
                  (256, 70), (300, 33)):
        if at < E:
            c[at] = n
    return c


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("E", [65, 130, 512])
@pytest.mark.parametrize("rows", [False, True])
def test_product(kind, E, rows, monkeypatch):
    monkeypatch.setitem(grouped.COUNTS, "many", counts_of(E))
    grouped.run_product(kind, "many", 136, 72, rows, rows, torch.float32 if rows else torch.bfloat16)


@pytest.mark.parametrize("E", [65, 130, 512])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)])
def test_wgrad(E, gather, dtype, accumulate, monkeypatch):
    monkeypatch.setitem(grouped.COUNTS, "many", counts_of(E))
    grouped.wgrad_case("many", 136, 72, gather, False, dtype, accumulate)


@pytest.mark.parametrize("name,N", [("one_row", 32776), ("two_of_three", 11016)])
def test_few_rows_of_wide_results(name, N):
    # enough tiles of 128 columns for every CU: the tile kernel takes few rows too
    grouped.run_product("fwd", name, N, 72, False, False, torch.bfloat16)


FEW = {
    (8, "two"): {1: 1, 6: 1},
    (8, "first_last"): {0: 2, 7: 3},
    (128, "edges"): {0: 1, 63: 2, 64: 1, 127: 20},
    (130, "past"): {64: 1, 128: 17, 129: 1},
    (512, "edges"): {0: 1, 63: 3, 64: 1, 255: 2, 256: 1, 320: 18, 511: 1},
    (512, "second_half"): {256: 1, 257: 1, 510: 2},
    (512, "last"): {511: 1},
}


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
@pytest.mark.parametrize("E,name", list(FEW))
@pytest.mark.parametrize("N,K", [(72, 256), (1096, 1280), (8200, 128)])
@pytest.mark.parametrize("rows", [False, True])
def test_w4_with_fewer_rows_than_experts(fmt, E, name, N, K, rows):
    if E * N * K > 1 << 29:
        N = 1 << 29 >> K.bit_length()
        N = N // E // 8 * 8
    say("w4 %s %d experts, %s, N=%d K=%d rows=%s" % (fmt, E, name, N, K, rows))
    few = FEW[(E, name)]
    counts = [few.get(e, 0) for e in range(E)]
    off, R = offsets_of(counts), sum(counts)
    assert R < E
    rng = np.random.default_rng([12, E, N, K])
    # experts without rows hold NaN scales (mxfp4) or NaN (int4): none of them is read into a result
    codes = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8))
    if fmt == "mxfp4":
        scales = torch.full((E, N, K // 32), 255, dtype=torch.uint8)
    else:
        scales = torch.full((E, N, K // 128), float("nan"), dtype=torch.bfloat16)
    for e in few:
        scales[e] = (torch.from_numpy(rng.integers(110, 135, scales.shape[1:], dtype=np.uint8)) if fmt == "mxfp4" else
                     torch.from_numpy(rng.uniform(0.001, 0.1, scales.shape[1:]).astype(np.float32)).to(torch.bfloat16))
    a = bf16(rng, R, K)
    ids = torch.from_numpy(rng.permutation(R).astype(np.int32)) if rows else None
    x = f64(a)[ids.numpy() // 2] if rows else f64(a)  # two grouped rows share a matrix row
    dev = None if ids is None else ids.to(DEV)
    out = Canvas(R, N, torch.float32)
    moe.grouped_gemm_w4(a.to(DEV), codes.to(DEV), scales.to(DEV), torch.from_numpy(off).to(DEV), out.t, a_rows=dev,
                        a_div=2, out_rows=dev)
    torch.cuda.synchronize()
    out.check_untouched(np.ones(R, dtype=bool))
    got = out.t[dev.long()] if rows else out.t
    for e in few:
        s = slice(off[e], off[e + 1])
        w = w4_values(codes[e:e + 1].numpy(), scales[e:e + 1], fmt)[0]
        mag, n = np.abs(w), K
        if fmt == "int4":  # (16 + q) - 24 inside the sum of a group of 128: terms up to 31 + 24 times |s x|
            mag, n = np.repeat(np.abs(f64(scales[e])), 128, axis=1) * 55, 128 + K // 128
        check(got[s], x[s] @ w.T, np.abs(x[s]) @ mag.T, n, "expert %d" % e)


def alternating(R, E):
    return [0 if i % 2 == 0 else R for i in range(E + 1)]


BAD = {
    "few_rows_wide": (60, 11016, [0, 50, 20, 60]),
    "decreasing": (700, 264, [700, 650, 300, 130, 0]),
    "outside": (700, 264, [-(1 << 31), 100, 90, (1 << 31) - 1, 350, 400, 700]),
    "overlapping": (700, 264, [0, 500, 100, 420, 40, 700]),
    # 20 experts of all 700 rows each: more tiles than 700 rows of 40 experts have
    "more_tiles_than_rows": (700, 264, alternating(700, 40)),
    "many_overlapping": (300, 136, alternating(300, 512)),
    "random": (700, 264, [int(v) for v in np.random.default_rng(3).integers(-300, 1000, 66)]),
}


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("name", list(BAD))
def test_offsets_that_no_routing_makes(kind, name):
    # every access stays inside the R rows, and a row that one expert alone claims comes out right, or, where the
    # experts claim more tiles than R rows have, is left as it was
    R, wide, bad = BAD[name]
    say("offsets %s %s" % (kind, name))
    E = len(bad) - 1
    rng = np.random.default_rng([8, R, E])
    N, K = (wide, 72) if kind == "fwd" else (72, wide)
    src, dst = (K, N) if kind == "fwd" else (N, K)
    a, w = bf16(rng, R, src), bf16(rng, E, N, K, scale=src ** -0.5)
    off = torch.from_numpy(np.array(bad, dtype=np.int64).astype(np.int32)).to(DEV)
    out = Canvas(R, dst, torch.bfloat16)
    call = moe.grouped_gemm if kind == "fwd" else moe.grouped_gemm_dgrad
    call(a.to(DEV), w.to(DEV), off, out.t)
    torch.cuda.synchronize()
    lo = np.clip(np.array(bad[:-1], dtype=np.int64), 0, R)
    hi = np.maximum(np.clip(np.array(bad[1:], dtype=np.int64), 0, R), lo)
    claims = sum(((np.arange(R) >= l) & (np.arange(R) < h)).astype(int) for l, h in zip(lo, hi))
    out.check_untouched(claims > 0)
    tiles = ((hi - lo) // 256 + ((hi - lo) % 256 > 128)).sum()
    W = f64(w)
    for e in range(E):
        alone = [i for i in range(lo[e], hi[e]) if claims[i] == 1]
        if alone and tiles <= R // 256 + E:
            m = W[e] if kind == "dgrad" else W[e].T
            check(out.t[torch.tensor(alone, device=DEV)], f64(a)[alone] @ m, np.abs(f64(a)[alone]) @ np.abs(m), src,
                  "expert %d" % e)
    got = f64(out.t)
    bound = np.abs(f64(a)).sum(1).max() * np.abs(W).max() + 8
    assert (np.abs(got) <= bound).all()  # sums of the rows' own values or the marker: nothing foreign
    dw = moe.grouped_gemm_wgrad(a.to(DEV), a.to(DEV), off)
    torch.cuda.synchronize()
    for e in range(E):
        x = f64(a)[lo[e]:hi[e]]
        check(dw[e], x.T @ x, np.abs(x).T @ np.abs(x), hi[e] - lo[e], "weight gradient of expert %d" % e)


@pytest.mark.parametrize("name", [n for n in BAD if n != "few_rows_wide"])
def test_w4_offsets_that_no_routing_makes(name):
    R, _, bad = BAD[name]
    say("w4 offsets %s" % name)
    E, N, K = len(bad) - 1, 72, 128
    rng = np.random.default_rng([9, R, E])
    a = bf16(rng, R, K)
    codes = torch.from_numpy(rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8))
    scales = torch.full((E, N, K // 32), 120, dtype=torch.uint8)
    out = Canvas(R, N, torch.float32)
    moe.grouped_gemm_w4(a.to(DEV), codes.to(DEV), scales.to(DEV),
                        torch.from_numpy(np.array(bad, dtype=np.int64).astype(np.int32)).to(DEV), out.t)
    torch.cuda.synchronize()
    lo = np.clip(np.array(bad[:-1], dtype=np.int64), 0, R)
    hi = np.maximum(np.clip(np.array(bad[1:], dtype=np.int64), 0, R), lo)
    claims = sum(((np.arange(R) >= l) & (np.arange(R) < h)).astype(int) for l, h in zip(lo, hi))
    out.check_untouched(claims > 0)
    w = w4_values(codes.numpy(), scales, "mxfp4")
    for e in range(E):
        alone = [i for i in range(lo[e], hi[e]) if claims[i] == 1]
        if alone:
            x = f64(a)[alone]
            check(out.t[torch.tensor(alone, device=DEV)], x @ w[e].T, np.abs(x) @ np.abs(w[e]).T, K, "expert %d" % e)
