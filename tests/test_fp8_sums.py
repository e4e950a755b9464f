"""What W4Q_FP8_SHORT goes with (no GPU needed)."""
import ctypes

import pytest
import torch

import w4a16_group_wise_amd as w4q
from test_block_abi import gemm
from w4a16_group_wise_amd import _lib


@pytest.mark.parametrize("dtype", [_lib.FP8_SHORT, 2 | _lib.FP8_SHORT, 1 | 2 * _lib.FP8_SHORT])
def test_short_sums_are_for_bf16(dtype):
    assert gemm(ydt=dtype) == w4q.W4Q_EINVAL
    n = ctypes.c_size_t(0)
    assert w4q.lib().fp8_gemm_workspace_size(100, 8, 256, dtype, ctypes.byref(n)) == w4q.W4Q_EINVAL


def test_workspace_of_bf16_results():
    for m, n, k in ((64, 4096, 4096), (65, 4096, 4096), (1531, 2050, 1152)):
        wide = w4q.workspace_size("fp8_gemm", m, n, k, 1)
        assert wide == w4q.workspace_size("fp8_gemm", m, n, k, 0)
        assert w4q.workspace_size("fp8_gemm", m, n, k, 1 | _lib.FP8_SHORT) <= wide or m <= 64
    # a workspace for short sums does not do for fp32's
    assert gemm(m=100, n=8, k=256, ydt=1, ws=4096, wb=w4q.workspace_size("fp8_gemm", 100, 8, 256, 1 | _lib.FP8_SHORT)) == w4q.W4Q_EINVAL


def test_short_sums_are_refused_for_fp32_results():
    x = torch.zeros(4, 128).to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        w4q.fp8_gemm(x, x, x, x, out_dtype=torch.float32, short_sums=True)
