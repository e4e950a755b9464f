"""The orthogonalised update is as exact as the same iteration in plain 32-bit products: held to a small
multiple of that iteration's own error, which a lost part of an operand exceeds by far (shown on the
CPU, by leaving parts out of an emulation)."""
import pytest
import torch

import layer_ref as R


def iterate(g, dtype=torch.float32, product=None, steps=5, eps=1e-7):
    """The iteration in `dtype` from X0 in 64 bits; product(x, y, transposed) in place of x @ y (x @ y^T)."""
    a, b, c = R.NS
    if product is None:
        def product(x, y, transposed):
            return x @ (y.mT.contiguous() if transposed else y)
    x = g.double() / (torch.linalg.vector_norm(g.double(), dim=(-2, -1), keepdim=True) + eps)
    flip = x.shape[-2] > x.shape[-1]
    x = (x.mT.contiguous() if flip else x).to(dtype)
    for _ in range(steps):
        t = product(x, x, True)
        x = a * x + product(b * t + c * product(t, t, False), x, False)
    return (x.mT.contiguous() if flip else x).double()


def excess(o, g, plain=None):
    """||o - exact|| over its bound, eight times the plain iteration's error and 2^-22 of the result.

    An operand in two fp16 parts is off by at most 2^-22, four times fp32's 2^-24, and a sum runs over three
    products a term (sqrt(3) times the roundings): below seven."""
    ref = iterate(g, torch.float64)
    plain = iterate(g) if plain is None else plain
    norm = torch.linalg.vector_norm(ref, dim=(-2, -1))
    bound = 8 * torch.linalg.vector_norm(plain - ref, dim=(-2, -1)) + 2.0 ** -22 * norm
    return (torch.linalg.vector_norm(o.double() - ref, dim=(-2, -1)) / bound).max()


def split(v):
    hi = (v * 8192).half()
    return hi.float(), (v * 8192 - hi.float()).half().float()


def emulated(keep):
    """Products of two fp16 parts in fixed point, of which only the pairs in `keep` are added."""
    def product(x, y, transposed):
        p, q = split(x), split(y.mT.contiguous() if transposed else y)
        return sum(p[i] @ q[j] for i, j in keep) * 2.0 ** -26
    return product


@pytest.mark.parametrize("r,c", [(129, 300), (256, 512), (300, 131)])
def test_a_lost_part_exceeds_the_bound(r, c):
    g = R.gradient(R.gen(r), 1, r, c)
    assert float(excess(iterate(g, product=emulated([(1, 0), (0, 1), (0, 0)])), g)) <= 1
    assert float(excess(iterate(g, product=emulated([(0, 0)])), g)) > 4             # no lo parts at all
    assert float(excess(iterate(g, product=emulated([(0, 1), (0, 0)])), g)) > 4     # the first operand's lost
    assert float(excess(iterate(g, product=emulated([(1, 0), (0, 0)])), g)) > 4     # the second one's
    assert float(excess(iterate(g.bfloat16().float(), product=lambda x, y, t: (
        x.bfloat16().float() @ (y.mT if t else y).bfloat16().float())), g.bfloat16().float())) > 4


# wide and tall, on tiles of 32, 64, 128 (alone, and two to a compute unit) and 256, whole and in ranges, and the
# short sides that iterate on square matrices
SHAPES = [(1, 256, 512), (1, 512, 256), (2, 65, 200), (1, 512, 520), (5, 300, 256), (1, 1100, 1300), (1, 1300, 1100),
          (1, 1100, 4500), (28, 1024, 1024), (1, 2048, 2048), (1, 2304, 1500), (1, 512, 8192), (1, 8192, 512),
          (1, 4096, 4128), (1, 4200, 3900), (1, 2500, 2900), (4, 64, 900), (1, 900, 31)]


@pytest.mark.gpu
@pytest.mark.parametrize("b,r,c", SHAPES)
def test_as_exact_as_plain_32_bit_products(dev, b, r, c):
    w4q = pytest.importorskip("w4a16_group_wise_amd")
    g = R.gradient(R.gen(b + r + c, dev), b, r, c, device=dev)
    plain = iterate(g)
    o = w4q.newton_schulz(g)
    assert float(excess(o, g, plain)) <= 1
    # the step's update on weights of zero is the same result
    w, m = torch.zeros_like(g), torch.zeros_like(g)
    w4q.muon_step(w, g, m, lr=1.0, momentum=0.0, nesterov=False, update_scale=1.0)
    assert torch.equal(-w, o)
