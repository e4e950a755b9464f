"""Gradients whose channels, tokens or operands differ by many powers of two from the tensor's largest
value, held to the bounds that the interface states (layer_bits.py)."""
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


@pytest.mark.parametrize("m,n,k", [(48, 41, 96), (200, 72, 160)])
@pytest.mark.parametrize("where", ["channels", "tokens", "inputs", "weights"])
@pytest.mark.parametrize("act,dtype", [("gelu", BF), ("silu", F32), ("relu", BF), ("none", F32), ("none", BF)])
def test_outliers(dev, m, n, k, where, act, dtype):
    x, w, scale, _ = R.layer(m, n, k, seed=m)
    w_hat = R.fake_quant_bf16(w, scale)
    gy = torch.randn(m, n, generator=R.gen(1)) * 1e-2
    z = torch.randn(m, n, generator=R.gen(2)).to(BF)

    def steps(count):  # one large, then 2^-1 .. 2^-40 of it
        return 2.0 ** -(torch.arange(count) % 41).float()
    if where == "channels":
        gy = gy * steps(n)
    elif where == "tokens":
        gy = gy * steps(m).view(-1, 1)
    elif where == "inputs":
        x = (x.float() * steps(k)).to(BF)
    else:
        w_hat = (w_hat.float() * steps(n).view(-1, 1)).to(BF)
    gy = gy.to(dtype)
    x, w_hat, gy, z = (t.to(dev) for t in (x, w_hat, gy, z))
    gx, gw, _ = w4q.lsq_linear_bwd(x, w_hat, gy, act=act, z=z if act != "none" else None)
    dx, dw, ex, ew = B.linear_bwd(x, w_hat, gy, z, act)
    within(gx, dx, R.stored(ex, dx, BF), "grad_x")
    within(gw, dw, R.stored(ew, dw, F32), "grad_w_hat")
