"""How many bits the sums of fp8_gemm keep."""
import pytest
import torch

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
F32 = torch.float32
E4 = torch.float8_e4m3fn


def equal(got, want, what):
    bad = got.double() != want
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m", [1, 13, 32, 40, 64, 200, 1531, 4096])
def test_bf16_results_have_the_sums_of_fp32(dev, m):
    """Eights of 256, -256 and six times 2^-6: 2^-14 of the largest, which sums of fp32 keep."""
    n, k = (4096 if m == 4096 else 300), 1024
    a = torch.full((m, k), 2.0 ** -6, device=dev)
    a[:, 0::8], a[:, 1::8] = 256.0, -256.0
    b = torch.ones(n, k, device=dev).to(E4)
    sa, sb = torch.ones(m, k // 128, device=dev), torch.ones(-(-n // 128), k // 128, device=dev)
    want = torch.full((m, n), 6 * k / 8 / 64, device=dev)   # 12, and no sum on the way needs more than 16 bits
    equal(w4q.fp8_gemm(a.to(E4), sa, b, sb), want.double(), "bf16")
    equal(w4q.fp8_gemm(a.to(E4), sa, b, sb, out_dtype=F32), want.double(), "fp32")
