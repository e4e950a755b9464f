"""grad_x from all bits of dz: short sums, where what dz lost would show in bf16 results, on every tile
size of the product (the output's sides choose it), ragged and odd ones included."""
import pytest
import torch

import layer_bits as B
import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
BF, F32 = torch.bfloat16, torch.float32


def within(got, ref, bound, what):
    err = (got.detach().double() - ref).abs()
    ok = err <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds, worst {float((err / bound).max()):.3g} of it"


# 64x64, 128x128 (alone, two to a compute unit) and 256x256 tiles; sums that end in the first stage and after it
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 40, 64), (64, 3, 96), (700, 16, 96), (515, 33, 288), (2048, 8, 2048),
                                   (2901, 17, 2912), (4500, 24, 4096)])
@pytest.mark.parametrize("act,dtype", [("relu", BF), ("none", F32), ("silu", BF), ("gelu", F32)])
def test_grad_x_takes_dz_in_22_bits(dev, m, n, k, act, dtype):
    x, w, scale, _ = R.layer(m, n, k, seed=m + n)
    w_hat = R.fake_quant_bf16(w, scale)
    # fp32 gradients and slopes fill dz's 24 bits
    gy = (1e-2 * torch.randn(m, n, generator=R.gen(1))).to(dtype)
    z = (2 * torch.randn(m, n, generator=R.gen(2))).to(BF)
    x, w_hat, gy, z = (t.to(dev) for t in (x, w_hat, gy, z))
    gx, gw, _ = w4q.lsq_linear_bwd(x, w_hat, gy, act=act, z=z if act != "none" else None)
    alone, _, _ = w4q.lsq_linear_bwd(x, w_hat, gy, act=act, z=z if act != "none" else None, with_w=False)
    assert torch.equal(alone, gx)
    dx, dw, ex, ew = B.linear_bwd(x, w_hat, gy, z, act)
    within(gx, dx, R.stored(ex, dx, BF), "grad_x")
    within(gw, dw, R.stored(ew, dw, F32), "grad_w_hat")
