"""The 4-bit products at the ends of their formats' ranges: every scale code of
MXFP4, and rows as large as the int4 form takes."""
import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV, E2M1, check, f64, offsets_of, w4_values

pytestmark = pytest.mark.gpu


def every_scale(K, group):
    """Weights [1, 4096, K] of MXFP4 that are zero but for the first of `group`:
    row 16 s + c has the code c under the scale s, and 127 under the others;
    and their values in 64 bits."""
    n = np.arange(4096)
    codes = np.zeros((1, 4096, K // 2), dtype=np.uint8)
    codes[0, :, 16 * group] = n % 16
    scales = np.full((1, 4096, K // 32), 127, dtype=np.uint8)
    scales[0, :, group] = n // 16
    v = np.where(n % 16 >= 8, -1.0, 1.0) * E2M1[n % 8] * 2.0 ** (n // 16 - 127.0)
    v = np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)  # past bf16 and fp32
    return codes, scales, np.where(n // 16 == 255, np.nan, v)


@pytest.mark.parametrize("counts", [[1], [16], [40]])
@pytest.mark.parametrize("K,group", [(32, 0), (96, 1), (512, 13), (6144, 190)])
def test_every_scale_of_mxfp4(counts, K, group):
    # one product of a weight and a power of two per result, which fp32 holds exactly
    say("MXFP4 scales, K=%d group=%d, %d rows" % (K, group, counts[0]))
    codes, scales, v = every_scale(K, group)
    rows = counts[0]
    for x in (1.0, 2.0 ** 50, -2.0 ** -20):
        a = torch.zeros(rows, K, dtype=torch.bfloat16)
        a[:, 32 * group] = x
        got = f64(moe.grouped_gemm_w4(a.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV),
                                      torch.from_numpy(offsets_of(counts)).to(DEV), out_dtype=torch.float32))
        want = v * x
        want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
        # below 2^-126 fp32 has steps of 2^-149
        tol = np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -150, 0.0)
        for r in range(rows):
            with np.errstate(invalid="ignore"):
                ok = (got[r] == want) | (np.isnan(got[r]) & np.isnan(want)) | (np.abs(got[r] - want) <= tol)
            assert ok.all(), (x, r, np.nonzero(~ok)[0][:4], got[r][~ok][:4], want[~ok][:4])


def test_a_nan_scale_stays_in_its_column():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (2, 72, 64), dtype=np.uint8)
    scales = rng.integers(120, 130, (2, 72, 4), dtype=np.uint8)
    scales[1, 5, 2] = 255
    a = torch.ones(20, 128, dtype=torch.bfloat16)
    y = moe.grouped_gemm_w4(a.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV),
                            torch.tensor([0, 9, 20], dtype=torch.int32, device=DEV))
    nan = torch.isnan(y).cpu()
    assert bool(nan[9:, 5].all()) and int(nan.sum()) == 11


@pytest.mark.parametrize("sign", ["same", "mixed", "halves"])
@pytest.mark.parametrize("K", [128, 640])
def test_int4_rows_below_2_to_116(sign, K):
    # the sum of a group, begun at -24 times the row's elements, passes fp32 nowhere: 24 * 128 * 2^116 < 2^128
    rng = np.random.default_rng([2, K])
    R, N = 5, 136
    x = np.full((R, K), (2.0 - 2.0 ** -7) * 2.0 ** 115)
    if sign == "mixed":
        x *= rng.choice([-1.0, 1.0], (R, K))
    if sign == "halves":
        x[:, 1::2] *= -1
    a = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    codes = rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    codes[0, 0], codes[0, 1], codes[0, 2], codes[0, 3] = 0x00, 0xFF, 0xF0, 0x0F
    scales = torch.from_numpy(rng.uniform(0.002, 0.01, (1, N, K // 128)).astype(np.float32)).to(torch.bfloat16)
    got = moe.grouped_gemm_w4(a.to(DEV), torch.from_numpy(codes).to(DEV), scales.to(DEV),
                              torch.tensor([0, R], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    w = w4_values(codes, scales, "int4")[0]
    # terms up to 31 + 24 times |s x| in a group of 128, then a sum over the groups
    mag = np.abs(f64(a)) @ (np.repeat(np.abs(f64(scales[0])), 128, axis=1) * 55).T
    check(got, f64(a) @ w.T, mag, 128 + K // 128, sign)
