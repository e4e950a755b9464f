"""fp8_gemm with short sums as it is used: side streams, captured graphs, buffers inside larger ones, results in place, numbers that
are none, offsets past 32 bits."""
import pytest
import torch

import block_ref as B
import layer_ref as R
from test_block_gpu import BF, GEMM_SIZES, operands, within
from test_block_use_gpu import inside, same
from w4a16_group_wise_amd import _lib

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
BYTES = 1 | _lib.FP8_SHORT


@pytest.mark.parametrize("m,n,k", GEMM_SIZES)
@pytest.mark.parametrize("square", [False, True])
def test_short_gemm(dev, m, n, k, square):
    fa, fb = (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2"))[(m + n) % 4]
    a, sa, b, sb = operands(dev, m, n, k, fa, fb, square, seed=m + n + k)
    g = R.gen(1, dev)
    bias, res = torch.randn(n, generator=g, device=dev), torch.randn(m, n, generator=g, device=dev).to(BF)
    for act in ("none", "gelu", "silu", "relu"):
        y = w4q.fp8_gemm(a, sa, b, sb, bias=bias, act=act, residual=res, short_sums=True)
        ref, err = B.gemm(a, sa, b, sb, bias, act, res, short=True)
        within(y, ref, err, act)


def calls(dev, seed):
    g = R.gen(seed, dev)
    out = {}
    for name, m, n, k in (("few", 5, 200, 1024), ("ranges", 300, 500, 8192), ("whole", 500, 500, 512), ("both", 1377, 6000, 2816)):
        a, sa, _, _ = w4q.fp8_quant(torch.randn(m, k, generator=g, device=dev))
        b, sb, _, _ = w4q.fp8_quant(torch.randn(n, k, generator=g, device=dev), square=True)
        bias, res = torch.randn(n, generator=g, device=dev), torch.randn(m, n, generator=g, device=dev).to(BF)
        # (codes travel as bytes: a copy of 8-bit floating point is one)
        out[name] = ((a.view(torch.uint8), sa, b.view(torch.uint8), sb, bias, res),
                     lambda i, ws: w4q.fp8_gemm(i[0].view(torch.float8_e4m3fn), i[1], i[2].view(torch.float8_e4m3fn), i[3], bias=i[4],
                                                act="silu", residual=i[5], short_sums=True, workspace=ws),
                     w4q.workspace_size("fp8_gemm", m, n, k, BYTES))
    return out


@pytest.mark.parametrize("name", ["few", "ranges", "whole", "both"])
def test_streams_repeats_and_workspaces(dev, name):
    inputs, call, bytes_ = calls(dev, 1)[name]
    want = call(inputs, None)
    assert same(call(inputs, None), want)
    if bytes_:
        ws = torch.full((bytes_ + 512,), 0xFF, dtype=torch.uint8, device=dev)   # what lies in scratch does not matter
        assert same(call(inputs, ws[:bytes_]), want) and bool((ws[bytes_:] == 0xFF).all())
    assert (bytes_ != 0) == (name in ("ranges", "both"))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for rep in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(call(inputs, None))
    torch.cuda.synchronize()
    assert all(same(o, want) for per in outs for o in per)


@pytest.mark.parametrize("name", ["few", "ranges", "whole", "both"])
def test_captured_and_replayed(dev, name):
    inputs, call, bytes_ = calls(dev, 1)[name]
    other, _, _ = calls(dev, 9)[name]
    ws = torch.empty(bytes_, dtype=torch.uint8, device=dev) if bytes_ else None
    static = tuple(t.clone() for t in inputs)
    call(static, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(static, ws)
    for rep in range(4):
        src = other if rep % 2 else inputs
        for s, t in zip(static, src):
            s.copy_(t)
        want = call(src, None)
        g.replay()
        torch.cuda.synchronize()
        assert same(out, want), f"replay {rep}"
        call(other, ws)


@pytest.mark.parametrize("d", [5, 96, 1001, 5496])
@pytest.mark.parametrize("rows", [7, 70, 513])
def test_nothing_beside_the_results_is_written(dev, d, rows):
    a, sa, _, _ = w4q.fp8_quant(torch.ones(rows, 300, device=dev))
    b, sb, _, _ = w4q.fp8_quant(torch.ones(d, 300, device=dev), square=True)
    out, kept = inside(torch.zeros(rows, d, dtype=BF, device=dev), dev, 7.0)
    w4q.fp8_gemm(a, sa, b, sb, out=out, short_sums=True)
    assert kept() and float((out.float() - 300).abs().max()) <= 300 * 2.0 ** -8


@pytest.mark.parametrize("m", [5, 200])
def test_codes_that_are_nan_and_scales_that_are_nan_stay_in_their_rows(dev, m):
    a, sa, b, sb = operands(dev, m, 150, 512, "e4m3", "e4m3", True)
    want = w4q.fp8_gemm(a, sa, b, sb, short_sums=True)
    a2, sa2 = a.clone(), sa.clone()
    a2.view(torch.uint8)[1, 300] = 0x7F
    sa2[3, 2] = float("nan")
    y = w4q.fp8_gemm(a2, sa2, b, sb, short_sums=True)
    ok = [i for i in range(m) if i not in (1, 3)]
    assert torch.equal(y[ok], want[ok]) and bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).all())
    sb2 = sb.clone()
    sb2[1, 0] = float("nan")
    y = w4q.fp8_gemm(a, sa, b, sb2, short_sums=True)
    assert torch.equal(y[:, :128], want[:, :128]) and bool(torch.isnan(y[:, 128:]).all())


@pytest.mark.parametrize("m,n,k", [(66000, 33000, 128), (40000, 130, 65536), (20, 40000, 65536)])
def test_past_32_bits(dev, m, n, k):
    # positive values, rows of different size: a row read from the wrong place shows
    def side(rows, seed):
        c = (torch.rand(rows, k, generator=R.gen(seed, dev), device=dev, dtype=BF) + 0.5).to(torch.float8_e4m3fn)
        s = (1 + torch.arange(rows, device=dev) % 97).float()[:, None] * torch.ones(1, k // 128, device=dev)
        return c, s.contiguous()
    (a, sa), (b, sb) = side(m, 1), side(n, 2)
    y = w4q.fp8_gemm(a, sa, b, sb, short_sums=True)
    for s in (slice(0, min(m, 7)), slice(m - min(m, 9), m)):
        for t in (slice(0, 11), slice(n - 13, n)):
            ref, err = B.gemm(a[s], sa[s], b[t], sb[t], short=True)
            within(y[s, t], ref, err, "y")


def test_short_sums_are_refused_for_fp32_results(dev):
    a, sa, b, sb = operands(dev, 8, 64, 256, "e4m3", "e4m3", True)
    with pytest.raises(ValueError, match="bf16"):
        w4q.fp8_gemm(a, sa, b, sb, out_dtype=torch.float32, short_sums=True)
