"""Plain 64-bit forms of the layer's product, its gradients and the orthogonalised update (test
infrastructure), with the error bounds the GPU results are held to.

Half steps (largest relative error of one rounding): bf16 2^-8, fp16 2^-11, fp32 2^-24.
"""
import math

import torch

H32, H16, HB = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8
GROUP = 32
ACTS = ("none", "relu", "gelu", "silu")
NS = (3.4445, -4.7750, 2.0315)
DACT_MAX = 1.13      # largest |act'|: gelu 1.1290, silu 1.0999


def codes(w, scale):
    d = scale.double().repeat_interleave(GROUP, dim=1)
    q = torch.round(w.double() / torch.where(d > 0, d, torch.ones_like(d))).clamp(-8, 7)
    return torch.where(d > 0, q, torch.zeros_like(q))


def fake_quant_bf16(w, scale):
    """bf16_RNE(fl32(scale * code)): both roundings are torch's own casts."""
    return (codes(w, scale).float() * scale.repeat_interleave(GROUP, dim=1)).to(torch.bfloat16)


def phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def act(z, name):
    return {"none": lambda: z, "relu": lambda: torch.where(z <= 0, torch.zeros_like(z), z),
            "gelu": lambda: z * phi(z), "silu": lambda: z * torch.sigmoid(z)}[name]()


def dact(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def linear_fwd(x, w_hat, bias, name, residual):
    """-> (z, y) in 64 bits, and the bound of |error| of each before it is stored.

    The sum of K exact products in fp32, in any order: at most (K + 1) 2^-24 of the sum of their
    magnitudes (bias included).  Through the activation: times |act'| <= 1.13, and its own evaluation
    (erfc, exp, a division and a few products: below 32 half steps of |z| + |y|)."""
    x, w = x.double(), w_hat.double()
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    ez = (x.shape[1] + 1) * H32 * mag
    y = act(z, name)
    ey = DACT_MAX * ez + (32 * H32 * (z.abs() + y.abs()) if name in ("gelu", "silu") else 0)
    if residual is not None:
        y = y + residual.double()
        ey = ey + H32 * (y.abs() + ey)
    return z, y, ez, ey


def linear_bwd(x, w_hat, grad_y, z, name):
    """-> (dz, dx, dw, db) in 64 bits and bounds of their errors, roundings to the outputs left out.

    dz itself: act' and the product, below 32 half steps of DACT_MAX |grad_y| (act' has terms of
    either sign, so the bound is not relative to dz).  With an activation or fp32 grad_y, dz enters dw
    in two fp16 parts (2^-22) and dx in one (2^-11), on a scale where its largest bound lies
    above 2^12, so that what falls below fp16's last step (2^-25) is 2^-37 of DACT_MAX max |grad_y|."""
    gy, xd, wd = grad_y.double(), x.double(), w_hat.double()
    split = name != "none" or grad_y.dtype == torch.float32
    dz = gy if name == "none" else gy * dact(z.double(), name)
    edz = torch.zeros_like(dz) if name in ("none", "relu") else 32 * H32 * DACT_MAX * gy.abs()
    fin = gy.abs()[torch.isfinite(gy)]
    floor = 2.0 ** -37 * DACT_MAX * (float(fin.max()) if fin.numel() else 0.0)
    eh = edz + (H16 * dz.abs() + floor if split else 0)
    el = edz + (2.0 ** -22 * dz.abs() + floor if split else 0)
    # x and W in fp16 (split): exact down to 2^-32 of the largest, an absolute 2^-38 of it below
    def aloss(t):
        return 2.0 ** -38 * float(t.abs()[torch.isfinite(t)].max()) if split else 0.0
    m, n = gy.shape
    dx, dw, db = dz @ wd, dz.t() @ xd, dz.sum(0)
    mx, mw = dz.abs() @ wd.abs(), dz.abs().t() @ xd.abs()
    # n (and 2 m) exact products summed in fp32
    ex = eh @ wd.abs() + (n + 1) * H32 * mx + dz.abs().sum(1, keepdim=True) * aloss(wd)
    ew = el.t() @ xd.abs() + (2 * m + 1) * H32 * mw + dz.abs().sum(0).unsqueeze(1) * aloss(xd)
    # column sums: at most 64 terms in fp32, then fp64
    eb = edz.sum(0) + 65 * H32 * dz.abs().sum(0) + H32 * db.abs()
    return dz, dx, dw, db, ex, ew, eb


def stored(e, y, dtype):
    """The bound with the rounding of the stored value (and, at the bottom, a subnormal's step)."""
    return e + (HB if dtype == torch.bfloat16 else H32) * (y.abs() + e) + (2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149)


def newton_schulz(g, steps=5, coeffs=NS, eps=1e-7):
    """-> (result in 64 bits, bound of the error in Frobenius norm).

    One step maps X to p(X), whose Frechet derivative is at most L = max |p'| = 3.9 on singular
    values up to 1.21.  In a step each product's operands are off by 2^-22 and its K-term fp32 sum
    by at most (3 K + 1) 2^-24 of the sum of magnitudes, taken here as sqrt(3 K) 2^-23 of the norms'
    product (rounding errors of either sign; entries of random sign): relative errors of A, A^2 and B X
    enter with weights |a| + |b| + |c| (times norms of A up to 1.46)."""
    a, b, c = coeffs
    x = g.double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    flip = x.shape[-2] > x.shape[-1]
    if flip:
        x = x.transpose(-2, -1)
    k = max(x.shape[-2], x.shape[-1])
    u = 2.0 ** -22 + math.sqrt(3 * k) * 2.0 ** -23
    lip = 3.9
    err = 2.0 ** -22 * torch.linalg.vector_norm(x, dim=(-2, -1))
    for _ in range(steps):
        nrm = torch.linalg.vector_norm(x, dim=(-2, -1))
        t = x @ x.transpose(-2, -1)
        x = a * x + (b * t + c * (t @ t)) @ x
        err = lip * err + 2 * (abs(a) + 1.46 * abs(b) + 1.46 ** 2 * abs(c)) * u * nrm
    if flip:
        x = x.transpose(-2, -1)
    return x, err


def gradient(gen, *shape, device="cpu"):
    """Gradients of a few strong directions above noise."""
    r = min(8, shape[-1], shape[-2])
    lead = shape[:-2]
    a = torch.randn(*lead, shape[-2], r, generator=gen, device=device)
    b = torch.randn(*lead, r, shape[-1], generator=gen, device=device)
    return 1e-3 * (a @ b + torch.randn(*shape, generator=gen, device=device))


def gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def layer(m, d_out, d_in, seed=0):
    """x bf16, w fp32, scale fp32, bias fp32 on the CPU."""
    g = gen(seed)
    x = (torch.randn(m, d_in, generator=g) * torch.exp(0.5 * torch.randn(d_in, generator=g))).to(torch.bfloat16)
    w = 0.02 * torch.randn(d_out, d_in, generator=g)
    amax = w.view(d_out, d_in // GROUP, GROUP).abs().amax(2)
    scale = (0.8 * amax / 7).to(torch.float16).float()
    return x, w, scale, 0.1 * torch.randn(d_out, generator=g)
