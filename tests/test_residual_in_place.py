"""The residual may be the output itself: no kernel that has an epilogue may promise the compiler that
nothing else reaches its output, and each gives the same bits in place."""
import os
import re

import pytest
import torch

import layer_ref as R

w4q = pytest.importorskip("w4a16_group_wise_amd")
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_group_wise_amd", "csrc")


def test_no_epilogue_kernel_restricts_its_output():
    seen = 0
    for f in sorted(os.listdir(CSRC)):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        # parameter lists of kernels and of the device functions that they store with
        for params in re.findall(r"__(?:global|device)__[^;{]*?\(([^{;]*W4Epilogue[^{;]*)\)\s*\{", src, flags=re.S):
            if re.search(r"\by\b", params):
                seen += 1
                assert not re.search(r"__restrict__\s+y\b", params), f
    assert seen >= 4


# the kernels of one row, of 2..16, of a tile per workgroup, of split sums and their fixup, and the written-out weights
@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,dq,scratch", [
    (1, 4096, 512, False, "all"), (1, 515, 96, False, "all"), (5, 9000, 512, False, "all"), (16, 300, 8192, False, "all"),
    (300, 515, 512, False, "none"), (4200, 2100, 96, False, "none"), (300, 515, 2048, False, "all"),
    (40, 700, 4096, False, "all"), (300, 515, 2048, True, "all"), (300, 515, 2048, True, "less"), (300, 515, 2048, True, "none"),
    (1600, 4200, 512, True, "all")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_gives_the_same_bits(dev, m, n, k, dq, scratch, dtype):
    x, w, scale, bias = (t.to(dev) for t in R.layer(m, n, k, seed=m))
    packed, s16 = w4q.quant_pack(w, scale)
    size = w4q.workspace_size("w4a16_linear", m, n, k, int(dq))
    product = w4q.workspace_size("w4a16_gemm_dq" if dq else "w4a16_gemm", m, n, k)
    ws = torch.empty({"all": size, "less": min(product, max(size - 256, 0)), "none": 0}[scratch], dtype=torch.uint8, device=dev)
    for act in ("none", "gelu"):
        res = torch.randn(m, n, generator=R.gen(3)).to(dtype).to(dev)
        kw = dict(bias=bias, act=act, dequant_bf16=dq, out_dtype=dtype, workspace=ws)
        want = w4q.w4a16_linear(x, packed, s16, residual=res.clone(), **kw)
        got = w4q.w4a16_linear(x, packed, s16, residual=res, out=res, **kw)
        assert got.data_ptr() == res.data_ptr() and torch.equal(got, want)
