"""fp8_gemm where every sum is exact: codes +-1, 1.5, 2, 3 and powers of two as scales, so that every term is a multiple of
2^-4 and no sum reaches 2^19, whatever its order.  Then fp32's sums round nothing, the 8-bit matrix cores' cut nothing
off (9 is the largest of eight products and 1/4 their last place, 2^-6 of it), and each result is the exact value rounded once:
equal bit for bit, which one code, scale or partial sum taken from the wrong place is not.  The sizes reach every kind of tile,
with and without split sums."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
BF, F32 = torch.bfloat16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def side(dev, rows, k, dtype, square, seed):
    """codes [rows][k], scales 2^-1, 1 or 2 for each row or 128 rows, and the values they stand for in 64 bits"""
    g = R.gen(seed, dev)
    c = torch.tensor([1, 1.5, 2, 3, -1, -1.5, -2, -3], device=dev)[torch.randint(0, 8, (rows, k), generator=g, device=dev)]
    n = -(-rows // 128) if square else rows
    s = torch.exp2(torch.randint(-1, 2, (n, k // 128), generator=g, device=dev).float())
    by_row = s.repeat_interleave(128, 0)[:rows] if square else s
    return c.to(dtype), s, c.double() * by_row.double().repeat_interleave(128, 1)


def parts(dev, m, n, k, square, fmts, seed=0):
    a, sa, x = side(dev, m, k, fmts[0], False, seed + 1)
    b, sb, w = side(dev, n, k, fmts[1], square, seed + 2)
    g = R.gen(seed + 3, dev)
    bias = torch.randint(-64, 65, (n,), generator=g, device=dev).float() / 4
    res = torch.randint(-64, 65, (m, n), generator=g, device=dev).float() / 4
    z = x @ w.t().contiguous()
    assert 9 * 4 * k < 2 ** 19 and bool((z * 16 == torch.round(z * 16)).all())
    return a, sa, b, sb, bias, res, z


def equal(got, want, what):
    want = want.float().to(got.dtype)   # (in 19 + 4 bits: the value itself in fp32)
    bad = got != want
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"


# few rows of 16, 32 and 64; tiles of 64, of 128 alone on a compute unit and two on one, of 256; split sums of each, also
# behind whole tiles: for bf16 values (the sums fp32's), codes (short sums), or both
SIZES = [(1, 130, 512), (13, 300, 1024), (16, 17, 8192), (29, 200, 640), (32, 1001, 2048), (33, 70, 1536), (64, 500, 2048), (65, 200, 384),
         (129, 1000, 512), (300, 257, 2048), (300, 500, 8192), (700, 900, 384), (513, 5496, 128), (518, 5443, 128), (1531, 2050, 1152),
         (837, 5827, 128), (67, 714, 10624), (193, 2008, 6784), (1797, 65, 8832), (1377, 6000, 2816), (4096, 4096, 512),
         (3222, 5011, 2304), (3390, 4785, 1152)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("square", [True, False])
def test_exact_sums(dev, m, n, k, square):
    fmts = ((E4, E4), (E5, E4), (E4, E5), (E5, E5))[(m + n + k // 128) % 4]
    a, sa, b, sb, bias, res, z = parts(dev, m, n, k, square, fmts, seed=m + n)
    equal(w4q.fp8_gemm(a, sa, b, sb, out_dtype=F32), z, "fp32")
    equal(w4q.fp8_gemm(a, sa, b, sb), z, "bf16")
    equal(w4q.fp8_gemm(a, sa, b, sb, short_sums=True), z, "bf16, short sums")
    y = torch.relu(z + bias.double()) + res.double()
    equal(w4q.fp8_gemm(a, sa, b, sb, bias=bias, act="relu", residual=res, out_dtype=F32), y, "fp32 with an epilogue")
    r16 = res.to(BF)
    for short in (False, True):
        equal(w4q.fp8_gemm(a, sa, b, sb, bias=bias, act="relu", residual=r16, short_sums=short), y, f"bf16 with an epilogue, short {short}")
        out = r16.clone()
        w4q.fp8_gemm(a, sa, b, sb, bias=bias, act="relu", residual=out, out=out, short_sums=short)
        equal(out, y, f"added in place, short {short}")


@pytest.mark.parametrize("fmts", [(E4, E4), (E5, E4), (E4, E5), (E5, E5)])
@pytest.mark.parametrize("m,n,k", [(5, 129, 512), (40, 129, 512), (200, 300, 512), (700, 2600, 256), (4096, 4096, 256)])
def test_every_pair_of_formats(dev, m, n, k, fmts):
    for square in (True, False):
        a, sa, b, sb, _, _, z = parts(dev, m, n, k, square, fmts)
        for short in (False, True):
            equal(w4q.fp8_gemm(a, sa, b, sb, short_sums=short), z, f"square {square}, short {short}")
