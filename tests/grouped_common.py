"""Shared helpers of the grouped-product and checkpoint tests: cases with
poisoned surroundings, references in 64 bits, and error bounds.

Bounds.  A product of n terms summed in fp32 in any order is off by at most
n * 2^-24 * sum|terms| to first order; the matrix unit may drop bits below
the largest term of a step, so twice that (n * 2^-23) is allowed, with 16
more terms for the joins of partial sums.  A result in bf16 is rounded once
more, by at most 2^-8 of its size.
"""
from __future__ import annotations

import numpy as np
import torch

DEV = torch.device("cuda:0")
BF16_STEP = 2.0 ** -8
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def sum_bound(n: int, absum: np.ndarray) -> np.ndarray:
    return (n + 16) * 2.0 ** -23 * absum


def bf16(rng, *shape, scale=1.0) -> torch.Tensor:
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()


def offsets_of(counts) -> np.ndarray:
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def poisoned(t: torch.Tensor, pad_cols: int = 0, value=float("nan")) -> torch.Tensor:
    """The [rows, width] CPU tensor as a strided view on the GPU whose padding
    columns hold `value`."""
    full = torch.full((t.shape[0], t.shape[1] + pad_cols), value, dtype=t.dtype, device=DEV)
    full[:, :t.shape[1]] = t.to(DEV)
    return full[:, :t.shape[1]]


class Canvas:
    """An output [rows, width] inside a larger buffer of a marker value: which
    elements were written, and that nothing else was."""

    MARK = {torch.bfloat16: -7.75, torch.float32: -7.75}

    def __init__(self, rows, width, dtype, pad_cols=8, guard_rows=3):
        self.g = guard_rows
        self.full = torch.full((rows + 2 * guard_rows, width + pad_cols), self.MARK[dtype], dtype=dtype, device=DEV)
        self.t = self.full[guard_rows:guard_rows + rows, :width]

    def check_untouched(self, written: np.ndarray):
        """Rows of `written` (bool [rows]) may hold anything inside the width;
        every other element still holds the marker."""
        mark = self.MARK[self.t.dtype]
        f = self.full.float().cpu().numpy()
        w = self.t.shape[1]
        assert (f[:, w:] == mark).all(), "columns past the width were written"
        assert (f[:self.g] == mark).all() and (f[f.shape[0] - self.g:] == mark).all(), "rows outside were written"
        assert (f[self.g:f.shape[0] - self.g, :w][~written] == mark).all(), "rows that belong to no expert were written"


def w4_values(codes: np.ndarray, scales: torch.Tensor, fmt: str) -> np.ndarray:
    """float64 [E,N,K] of 4-bit codes uint8 [E,N,K/2] and their scales."""
    q = np.empty(codes.shape[:2] + (2 * codes.shape[2],), dtype=np.int64)
    q[:, :, 0::2], q[:, :, 1::2] = codes & 15, codes >> 4
    if fmt == "mxfp4":
        v = np.where(q >= 8, -1.0, 1.0) * E2M1[q & 7]
        s = 2.0 ** (scales.numpy().astype(np.float64) - 127)
        return v * np.repeat(s, 32, axis=2)
    return (q - 8.0) * np.repeat(f64(scales), 128, axis=2)


def check(got: torch.Tensor, ref: np.ndarray, absum: np.ndarray, n: int, what: str = ""):
    """Elementwise bound of a sum of n terms, rounded to got's type."""
    g = f64(got)
    tol = sum_bound(n, absum)
    if got.dtype == torch.bfloat16:
        tol = tol + BF16_STEP * (np.abs(ref) + tol)
    bad = ~(np.abs(g - ref) <= tol + 1e-30)
    assert not bad.any(), "%s: %d of %d off, first at %s: %r for %r (bound %r)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], ref[bad][0], tol[bad][0])
