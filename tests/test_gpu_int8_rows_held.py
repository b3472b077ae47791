"""Products in 8-bit integers of bf16 rows that are not all held: one process's share of the experts."""
import ctypes

import numpy as np
import pytest
import torch

import moe_layer_align_amd as moe
from gpu_common import say
from grouped_common import DEV, bf16
from test_abi_tokens import GroupedInt8Args

pytestmark = pytest.mark.gpu


def product(a, w, scale, off, out, work, R):
    """moe_grouped_gemm_int8 of bf16 rows, by the C entry point."""
    E, N, K = w.shape

    def rows(t):
        return moe._Rows(t.data_ptr(), t.stride(0), t.shape[0], 1, None)

    args = GroupedInt8Args(R, E, N, K, off.data_ptr(), rows(a), None, w.data_ptr(), scale.data_ptr(), rows(out), 0,
                           work.data_ptr(), work.numel())
    f = moe.load().moe_grouped_gemm_int8
    f.argtypes = [ctypes.POINTER(GroupedInt8Args), ctypes.c_void_p]
    assert f(ctypes.byref(args), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()


# streamed in few passes, and in tiles; codes by one wave, four and sixteen a row
@pytest.mark.parametrize("N,K", [(24, 144), (2056, 2064), (64, 16400)])
@pytest.mark.parametrize("counts", [[100, 0, 150, 50], [0, 0, 0, 0], [1, 0, 0, 0], [250, 250, 250, 250]])
@pytest.mark.parametrize("more", [0, 77])
def test_rows_behind_the_experts_are_not_read(N, K, counts, more):
    say("bf16 rows held: N=%d K=%d %s" % (N, K, counts))
    R, E = 1000, len(counts)
    rng = np.random.default_rng([N, K, counts[0]])
    n = sum(counts)
    a = bf16(rng, R + more, K).to(DEV)  # `more`: a matrix of more rows than are grouped
    a[n:] = float("nan")
    w = torch.from_numpy(rng.integers(-127, 128, (E, N, K), dtype=np.int8)).to(DEV)
    scale = torch.from_numpy(rng.random((E, N)).astype(np.float32)).to(DEV)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    size = moe.load().moe_grouped_int8_workspace_size(R, E, N, K, R + more)
    at = ((R + more) * K + 255) // 256 * 256  # of the scales, behind the codes
    assert size == at + 4 * (R + more)
    work = torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV)
    product(a, w, scale, off, out, work, R)
    codes, scales = moe.quant_int8(a[:n].contiguous())
    assert torch.equal(work[:n * K].view(torch.int8).view(n, K), codes)
    assert torch.equal(work[at:at + 4 * n].view(torch.float32), scales)
    # nothing was made of the other rows
    assert bool((work[n * K:at] == 0x5A).all()) and bool((work[at + 4 * n:] == 0x5A).all())
    full, fs = torch.zeros(R, K, dtype=torch.int8, device=DEV), torch.zeros(R, device=DEV)
    full[:n], fs[:n] = codes, scales
    want = moe.grouped_gemm_int8(full, w, scale, off, torch.full_like(out, 7.0), a_scale=fs)
    assert torch.equal(out, want) and bool((out[n:] == 7).all())
