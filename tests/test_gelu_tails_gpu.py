"""gelu and its derivative to fp32's digits of themselves, far out on the negative side too, in every
kernel that applies them.  Activations of zero make z the bias exactly."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
BF, F32 = torch.bfloat16, torch.float32

# Phi(z) for z <= 0 in fp32, in half steps: 1 / (1 + p |z|) by an addition and a reciprocal (1 + 2), a polynomial
# in it (below 4, its own error 0.4), exp(-z^2 / 2) (2 for 2^x, 2 for its two-part exponent), two products
# (2): below 14; times z and stored 2 more.  1 - Phi and the sum in the derivative add less.
REL = 16 * R.H32
# the hardware's 2^x gives 0 below 2^-126: there z Phi(z) is below 2^-127 (Phi is 0.03 of exp(-z^2 / 2) at -13.2)
FLOOR = 2.0 ** -127


def points(n):
    """n values of z: the tails, the ordinary range and values next to 0, fp32."""
    g = R.gen(n)
    t = torch.cat((torch.linspace(-14.5, 14.5, n - n // 3, dtype=torch.float64),
                   torch.exp(torch.linspace(-40, 0, n // 3, dtype=torch.float64)) * torch.randn(n // 3, generator=g).sign()))
    return t[torch.randperm(n, generator=g)].float()


def tail(z):
    """z Phi(z) in 64 bits (erfc keeps its digits)."""
    z = z.double()
    return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))


def within(got, ref, bound, what):
    err = (got.detach().cpu().double() - ref).abs()
    ok = err <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds, worst {float((err / bound).max()):.3g} of it"


def test_reference_keeps_its_digits():
    # Phi(-x) between its published bounds phi(x) (1/x - 1/x^3) and phi(x) / x
    z = -torch.linspace(4, 14.5, 1000, dtype=torch.float64)
    phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    t = tail(z) / z
    assert bool((t < phi / -z).all()) and bool((t > phi * (1 / -z + 1 / z ** 3)).all())


@pytest.mark.parametrize("n", [4096, 2051])
@pytest.mark.parametrize("m", [1, 3, 40])
def test_gelu_of_the_layers(dev, m, n):
    z = points(n)
    ref = tail(z).expand(m, n)
    x = torch.zeros(m, 256, dtype=BF, device=dev)
    w = 0.02 * torch.randn(n, 256, generator=R.gen(1)).to(dev)
    scale = torch.full((n, 8), 0.01, device=dev)
    packed, s16 = w4q.quant_pack(w, scale)
    b = z.to(dev)
    for dtype, half in ((F32, 0.0), (BF, R.HB)):
        bound = (REL + half * (1 + REL)) * ref.abs() + FLOOR
        y, _, _ = w4q.lsq_linear_fwd(x, w, scale, bias=b, act="gelu", out_dtype=dtype)
        within(y, ref, bound, f"lsq_linear_fwd {dtype}")
        for dq in (False, True):
            y = w4q.w4a16_linear(x, packed, s16, bias=b, act="gelu", dequant_bf16=dq, out_dtype=dtype)
            within(y, ref, bound, f"w4a16_linear {dtype} dq={dq}")


@pytest.mark.parametrize("n", [4096, 2051])
def test_gelu_derivative(dev, n):
    # one row and a gradient of 1: grad_bias is the derivative itself
    z = points(n).to(BF)
    zd = z.double()
    terms = 0.5 * torch.erfc(zd.abs() / math.sqrt(2.0)), zd * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    cdf = torch.where(zd < 0, terms[0], 1 - terms[0])
    _, _, gb = w4q.lsq_linear_bwd(torch.zeros(1, 32, dtype=BF, device=dev), torch.zeros(n, 32, dtype=BF, device=dev),
                                  torch.ones(1, n, dtype=F32, device=dev), act="gelu", z=z.view(1, n).to(dev), with_x=False,
                                  with_w=False, with_bias=True)
    # the terms have opposite signs for z < 0, so the bound is relative to both; 13.2 2^-126 0.4 where 2^x gives 0
    within(gb, cdf + terms[1], REL * (cdf + terms[1].abs()) + 2.0 ** -123, "grad_bias")
