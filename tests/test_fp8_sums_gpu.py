"""How many bits the sums of fp8_gemm keep."""
import pytest
import torch

import layer_ref as R

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


def cut_off(a, sa, b, sb):
    """What short sums may lose, in 64 bits.  A code has 4 bits, so a product 8: its last place is 2^-8 of it or more.  Of an eight's
    products those of 2^-5 of the largest and more reach no lower than 2^-13 of it and lose nothing; one below loses less than
    2^-13 of the largest, and never more than itself.  (On normal values about a ninth of 7 2^-13 of all magnitudes.)"""
    k = a.shape[1]
    p = (a.float()[:, None, :] * b.float()[None, :, :]).double().abs()      # exact: 8 bits
    p = p.view(*p.shape[:2], -1, 8)
    top = p.amax(dim=3, keepdim=True)
    lost = torch.where(p < 2.0 ** -5 * top, torch.minimum(p, 2.0 ** -13 * top), torch.zeros((), dtype=torch.float64, device=p.device))
    factor = (sa[:, None, :].double() * sb[None, :, :].double()).abs()
    mag = p.view(*p.shape[:2], k // 128, 128).sum(3) * factor
    return (lost.sum(3).view(*p.shape[:2], k // 128, 16).sum(3) * factor).sum(2), mag.sum(2)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("square", [True, False])
@pytest.mark.parametrize("m,n,k", [(13, 300, 12288), (64, 500, 12288), (200, 700, 12288), (1531, 2050, 4096), (4096, 4096, 4096)])
def test_short_sums_lose_what_the_matrix_cores_cut(dev, m, n, k, square, fmt):
    g = R.gen(m + k, dev)
    x = torch.randn(m, k, generator=g, device=dev) * torch.exp(0.5 * torch.randn(k, generator=g, device=dev))
    w = 0.02 * torch.randn(n, k, generator=g, device=dev)
    a, sa, _, _ = w4q.fp8_quant(x, fmt=fmt)
    b, sb, _, _ = w4q.fp8_quant(w, square=square)
    short = w4q.fp8_gemm(a, sa, b, sb, short_sums=True)
    rows = torch.randperm(m, generator=torch.Generator().manual_seed(1))[:8].to(dev)
    cols = torch.randperm(n, generator=torch.Generator().manual_seed(2))[:32].to(dev)
    sbc = sb[cols // 128] if square else sb[cols]
    av, bv, sav = a.float()[rows], b.float()[cols], sa[rows]
    ref = (av.double() * sav.double().repeat_interleave(128, 1)) @ (bv.double() * sbc.double().repeat_interleave(128, 1)).t().contiguous()
    lost, mag = cut_off(av, sav, bv, sbc)
    # a block's factor and the sums: k + 6 roundings of fp32 at most, as without the cut
    bound = lost + (k + 6) * 2.0 ** -24 * mag
    err = (short[rows][:, cols].double() - ref).abs()
    half = 2.0 ** -8 * (ref.abs() + bound)
    assert bool((err <= bound + half).all()), f"worst {float((err / (bound + half)).max()):.3g} of the bound"
