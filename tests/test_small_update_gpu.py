"""The orthogonalised update keeps the digits of 32-bit products where the input is far below eps, and
with every tile size and layout of the products."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
F32 = torch.float32


def iterate(g, dtype, steps=5, eps=1e-7, coeffs=R.NS):
    """The iteration in `dtype` from X0 in 64 bits."""
    a, b, c = coeffs
    x = g.double() / (torch.linalg.vector_norm(g.double(), dim=(-2, -1), keepdim=True) + eps)
    flip = x.shape[-2] > x.shape[-1]
    x = (x.mT.contiguous() if flip else x).to(dtype)
    for _ in range(steps):
        t = x @ x.mT.contiguous()
        x = a * x + (b * t + c * (t @ t)) @ x
    x = x.double()
    return x.mT.contiguous() if flip else x


def near_fp32(o, g, what, **kw):
    """The result's error is at most eight times that of the same iteration in plain fp32.  An operand in two
    fp16 parts is off by at most 2^-22, four times fp32's 2^-24, and a sum runs over three products a term
    (sqrt(3) times the roundings): below seven.  2^-22 of the result where the plain form happens to be exact."""
    ref = iterate(g, torch.float64, **kw)
    norm = torch.linalg.vector_norm(ref, dim=(-2, -1))
    plain = torch.linalg.vector_norm(iterate(g, torch.float32, **kw) - ref, dim=(-2, -1))
    err = torch.linalg.vector_norm(o.double() - ref, dim=(-2, -1))
    bound = 8 * plain + 2.0 ** -22 * norm
    assert bool((err <= bound).all()), f"{what}: {(err / bound).max():.3g} of the bound, {(err / norm).max():.3g} of the result"


SHAPES = [(1, 40, 200), (3, 90, 33), (1, 70, 90), (1, 256, 512), (1, 300, 131), (2, 130, 777), (1, 1100, 1300)]


@pytest.mark.parametrize("b,r,c", SHAPES)
@pytest.mark.parametrize("norm", [1e-2, 1e-5, 1e-7, 1e-9, 1e-12, 1e-20, 1e-33])
def test_inputs_far_below_eps(dev, b, r, c, norm):
    g = R.gradient(R.gen(b + r, dev), b, r, c, device=dev)
    g = (g.double() * (norm / torch.linalg.vector_norm(g.double(), dim=(-2, -1), keepdim=True))).float()
    near_fp32(w4q.newton_schulz(g), g, f"norm {norm}")
    # the step on weights of zero is the update itself, times -lr
    w, m = torch.zeros_like(g), torch.zeros_like(g)
    w4q.muon_step(w, g, m, lr=1.0, momentum=0.0, nesterov=False, update_scale=1.0)
    assert torch.equal(-w, w4q.newton_schulz(g))


def test_batches_of_mixed_sizes(dev):
    # each matrix of a batch has its own power of two
    g = R.gradient(R.gen(3, dev), 6, 200, 150, device=dev)
    s = torch.tensor([1.0, 1e-12, 0.0, 1e-8, 1e4, 1e-30], device=dev).view(6, 1, 1)
    o = w4q.newton_schulz(g * s)
    keep = [0, 1, 3, 4, 5]
    near_fp32(o[keep], (g * s)[keep], "batch")
    assert bool((o[2] == 0).all())
    for i in keep:
        near_fp32(w4q.newton_schulz((g * s)[i].contiguous()), (g * s)[i], f"matrix {i}")


@pytest.mark.parametrize("coeffs,steps", [((1.5, -0.5, 0.0), 20), ((1.875, -1.25, 0.375), 12), (R.NS, 1), (R.NS, 9)])
def test_other_coefficients_far_below_eps(dev, coeffs, steps):
    # small singular values grow through the steps, some of them to 1
    g = R.gradient(R.gen(7, dev), 1, 140, 220, device=dev)
    for norm in (1e-9, 1e-12):
        t = (g.double() * (norm / torch.linalg.vector_norm(g.double()))).float()
        near_fp32(w4q.newton_schulz(t, coeffs=coeffs, steps=steps), t, f"norm {norm}", coeffs=coeffs, steps=steps)
