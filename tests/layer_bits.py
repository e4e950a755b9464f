"""Bounds and plain forms that go beyond layer_ref.py's: what the operands' bits leave of each result
(test infrastructure).  Half steps as there: bf16 2^-8, fp16 2^-11, fp32 2^-24."""
import torch

import layer_ref as R


def linear_bwd(x, w_hat, grad_y, z, name):
    """-> (dx, dw) in 64 bits and bounds of their errors, the roundings to the outputs left out.

    With gelu, silu or fp32 grad_y, dz = grad_y act' enters both products in two fp16 parts of dz 2^e, with
    2^e max|grad_y| in [2^13, 2^14): hi = RNE(s), lo = RNE(s - hi), |s - hi| <= 2^-11 |s|, so lo is off by
    2^-22 |s|, or, where it is subnormal, by half of fp16's last step, 2^-25, which is at most 2^-38 of
    max|grad_y|.  x and W enter as one fp16 value times a power of two that brings their largest to [2^13,
    2^14): 8 bits, so the last one lies above 2^-24 from 2^-30 of the largest on; below, half a step is at
    most 2^-38 of it.  Otherwise dz is grad_y or 0, and all enter as they are.  dz itself, where it is
    not exact: 32 half steps of 1.13 |grad_y|.  n (m) exact products of each part summed in fp32: 2 n + 1
    half steps of the magnitudes' sum."""
    gy, xd, wd = grad_y.double(), x.double(), w_hat.double()
    split = name in ("gelu", "silu") or grad_y.dtype == torch.float32
    dz = gy if name == "none" else gy * R.dact(z.double(), name)
    edz = torch.zeros_like(dz)
    if name in ("gelu", "silu"):
        edz = 32 * R.H32 * R.DACT_MAX * gy.abs()

    def top(t):
        t = t.abs()[torch.isfinite(t)]
        return float(t.max()) if t.numel() else 0.0
    e = edz + (2.0 ** -22 * dz.abs() + 2.0 ** -38 * top(gy) if split else 0)
    m, n = gy.shape
    dx, dw = dz @ wd, dz.t() @ xd
    mx, mw = dz.abs() @ wd.abs(), dz.abs().t() @ xd.abs()
    loss = 2.0 ** -38 if split else 0.0
    ex = e @ wd.abs() + (2 * n + 1) * R.H32 * mx + dz.abs().sum(1, keepdim=True) * (loss * top(wd))
    ew = e.t() @ xd.abs() + (2 * m + 1) * R.H32 * mw + dz.abs().sum(0).unsqueeze(1) * (loss * top(xd))
    return dx, dw, ex, ew
