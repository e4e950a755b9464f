"""Host-side checks of the layer's C ABI and its binding (no GPU needed): every declared function is
exported and bound, and bad arguments are refused before anything reaches the device."""
import ctypes
import os
import re

import pytest
import torch

import layer_ref as R
import w4a16_group_wise_amd as w4q
from w4a16_group_wise_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B = 4096, 4097  # fake addresses, aligned and misaligned: never dereferenced, the checks fail first
INV, SHAPE, ALIGN, UNSUP = w4q.W4Q_EINVAL, w4q.W4Q_ESHAPE, w4q.W4Q_EALIGN, w4q.W4Q_EUNSUPPORTED


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "w4a16q_layer.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\**(\w+)\s*\(", src, flags=re.M))
    assert names == set(_lib.LAYER_SIGNATURES)
    l = ctypes.CDLL(_lib.LIB_PATH)
    for n in names:
        assert hasattr(l, n), n
    assert not names & set(_lib.SIGNATURES)


def fwd(**kw):
    a = dict(x=A, m=4, w=A, scale=A, d_out=8, d_in=64, bias=None, act=0, res=None, w_hat=A, z=None, y=A, ydt=1, ws=None, wb=0)
    a.update(kw)
    return w4q.lib().lsq_linear_fwd(a["x"], a["m"], a["w"], a["scale"], a["d_out"], a["d_in"], a["bias"], a["act"], a["res"],
                                    a["w_hat"], a["z"], a["y"], a["ydt"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(w_hat=None), INV), (dict(y=None), INV), (dict(w=None), INV), (dict(scale=None), INV),
    (dict(act=4), INV), (dict(act=-1), INV), (dict(ydt=2), INV), (dict(m=0), SHAPE), (dict(d_out=0), SHAPE),
    (dict(d_in=0), SHAPE), (dict(d_in=48), SHAPE), (dict(m=1 << 41), SHAPE), (dict(d_in=32 << 17), UNSUP),
    (dict(m=1 << 30, d_in=32, d_out=1), UNSUP), (dict(m=1 << 24, d_out=1 << 14, d_in=1 << 14), UNSUP),
    (dict(m=(1 << 30) - 1, d_in=32, d_out=1), UNSUP), (dict(m=1 << 29, d_in=32, d_out=128), UNSUP),
    (dict(x=A + 2), ALIGN), (dict(w=A + 4), ALIGN), (dict(w_hat=A + 8), ALIGN), (dict(scale=A + 2), ALIGN),
    (dict(bias=A + 1), ALIGN), (dict(y=B), ALIGN), (dict(ydt=0, y=A + 2), ALIGN), (dict(res=B), ALIGN),
    (dict(ydt=0, res=A + 2), ALIGN), (dict(z=B), ALIGN), (dict(ws=None, wb=256), INV), (dict(ws=A + 128, wb=256), ALIGN)])
def test_linear_fwd_refusals(kw, want):
    assert fwd(**kw) == want


def bwd(**kw):
    a = dict(x=A, m=4, w_hat=A, d_out=8, d_in=64, gy=A, gdt=1, act=3, z=A, gx=A, gw=A, gb=A, ws=A, wb=1 << 30)
    a.update(kw)
    return w4q.lib().lsq_linear_bwd(a["x"], a["m"], a["w_hat"], a["d_out"], a["d_in"], a["gy"], a["gdt"], a["act"], a["z"],
                                    a["gx"], a["gw"], a["gb"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(w_hat=None), INV), (dict(gy=None), INV), (dict(z=None), INV), (dict(act=9), INV),
    (dict(gdt=2), INV), (dict(gx=None, gw=None, gb=None), INV), (dict(m=-1), SHAPE), (dict(d_in=33), SHAPE),
    (dict(d_out=-3), SHAPE), (dict(m=4194241), UNSUP), (dict(d_in=32 << 17), UNSUP), (dict(d_out=(1 << 20) + 1), UNSUP),
    (dict(m=4194240, d_out=1 << 14, d_in=32), UNSUP), (dict(x=A + 8), ALIGN),
    (dict(w_hat=A + 8), ALIGN), (dict(gy=A + 8), ALIGN), (dict(z=B), ALIGN), (dict(gx=B), ALIGN), (dict(gw=A + 2), ALIGN),
    (dict(gb=A + 2), ALIGN), (dict(ws=None, wb=0), INV), (dict(ws=A + 16), ALIGN), (dict(wb=1024), INV)])
def test_linear_bwd_refusals(kw, want):
    assert bwd(**kw) == want


def w4(**kw):
    a = dict(x=A, m=4, p=A, s=A, d_out=8, d_in=64, bias=None, act=0, res=None, y=A, ydt=0, mode=0, ws=None, wb=0)
    a.update(kw)
    return w4q.lib().w4a16_linear(a["x"], a["m"], a["p"], a["s"], a["d_out"], a["d_in"], a["bias"], a["act"], a["res"],
                                  a["y"], a["ydt"], a["mode"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INV), (dict(p=None), INV), (dict(s=None), INV), (dict(y=None), INV), (dict(act=4), INV),
    (dict(ydt=3), INV), (dict(mode=2), INV), (dict(m=0), SHAPE), (dict(d_in=40), SHAPE), (dict(d_out=0), SHAPE),
    (dict(mode=1), UNSUP), (dict(mode=1, m=300, d_in=320), UNSUP), (dict(m=1, d_in=32 << 20), UNSUP),
    (dict(x=A + 2), ALIGN), (dict(p=A + 8), ALIGN), (dict(s=B), ALIGN), (dict(y=A + 2), ALIGN), (dict(bias=A + 2), ALIGN),
    (dict(res=A + 2), ALIGN), (dict(ws=None, wb=1), INV), (dict(ws=A + 64, wb=1 << 20), ALIGN)])
def test_w4a16_linear_refusals(kw, want):
    assert w4(**kw) == want


def ns(**kw):
    a = dict(g=A, gdt=0, b=1, r=8, c=8, steps=5, co=R.NS, eps=1e-7, out=A, odt=0, ws=A, wb=1 << 40)
    a.update(kw)
    co = None if a["co"] is None else (ctypes.c_float * 3)(*a["co"])
    return w4q.lib().newton_schulz(a["g"], a["gdt"], a["b"], a["r"], a["c"], a["steps"], co, a["eps"], a["out"], a["odt"],
                                   a["ws"], a["wb"], None)


NS_BAD = [
    (dict(steps=0), INV), (dict(steps=65), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(co=(4.0, 0.0, 0.0)), INV), (dict(co=(0.0, 9.0, 0.0)), INV),
    (dict(co=(float("nan"), 0.0, 0.0)), INV), (dict(co=(3.4445, -4.775, 4.0)), INV), (dict(b=0), SHAPE), (dict(r=0), SHAPE),
    (dict(c=-1), SHAPE), (dict(b=65536), UNSUP), (dict(r=131073), UNSUP), (dict(c=131073), UNSUP),
    (dict(b=65535, r=4096, c=4096), UNSUP), (dict(ws=None, wb=0), INV), (dict(ws=A + 128), ALIGN), (dict(wb=100), INV)]


@pytest.mark.parametrize("kw,want", NS_BAD + [
    (dict(g=None), INV), (dict(out=None), INV), (dict(co=None), INV), (dict(gdt=2), INV), (dict(odt=-1), INV),
    (dict(g=A + 2), ALIGN), (dict(out=A + 2), ALIGN), (dict(g=B, gdt=1), ALIGN)])
def test_newton_schulz_refusals(kw, want):
    assert ns(**kw) == want


def muon(**kw):
    a = dict(w=A, g=A, m=A, b=1, r=8, c=8, lr=0.02, mu=0.95, wd=0.0, sc=1.0, co=R.NS, nes=1, steps=5, eps=1e-7, ws=A, wb=1 << 40)
    a.update(kw)
    hp = _lib.MuonParams(a["lr"], a["mu"], a["wd"], a["sc"], (ctypes.c_float * 3)(*a["co"]), a["nes"], a["steps"], a["eps"])
    return w4q.lib().muon_step(a["w"], a["g"], a["m"], a["b"], a["r"], a["c"], ctypes.byref(hp), a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,want", NS_BAD + [
    (dict(w=None), INV), (dict(g=None), INV), (dict(m=None), INV), (dict(lr=-1.0), INV), (dict(lr=float("nan")), INV),
    (dict(mu=1.0), INV), (dict(mu=-0.1), INV), (dict(mu=float("nan")), INV), (dict(wd=-1.0), INV),
    (dict(sc=float("inf")), INV), (dict(nes=2), INV), (dict(w=A + 2), ALIGN), (dict(g=A + 2), ALIGN), (dict(m=A + 2), ALIGN)])
def test_muon_refusals(kw, want):
    assert muon(**kw) == want
    assert w4q.lib().muon_step(A, A, A, 1, 8, 8, None, A, 1 << 40, None) == INV


def test_workspace_queries():
    L, n = w4q.lib(), ctypes.c_size_t(0)
    p = ctypes.byref(n)
    assert L.lsq_linear_fwd_workspace_size(4, 8, 64, None) == INV
    assert L.lsq_linear_fwd_workspace_size(0, 8, 64, p) == SHAPE
    assert L.lsq_linear_bwd_workspace_size(4, 8, 48, 1, 0, p) == SHAPE
    assert L.lsq_linear_bwd_workspace_size(4, 8, 64, 2, 0, p) == INV
    assert L.w4a16_linear_workspace_size(4, 8, 64, 0, None) == INV
    assert L.w4a16_linear_workspace_size(4, 8, 64, 2, p) == INV
    assert L.w4a16_linear_workspace_size(4, 8, 65, 0, p) == SHAPE
    assert L.newton_schulz_workspace_size(1, 0, 8, p) == SHAPE
    assert L.newton_schulz_workspace_size(1, 8, 131073, p) == UNSUP
    assert w4q.workspace_size("lsq_linear_fwd", 1, 32, 32) == 0
    assert w4q.workspace_size("newton_schulz", 1, 64, 64) > 0
    assert (w4q.workspace_size("newton_schulz", 2, 512, 256) > w4q.workspace_size("newton_schulz", 1, 512, 256))
    # two fp16 parts of dz with an activation
    assert w4q.workspace_size("lsq_linear_bwd", 512, 512, 512, 1, 3) > w4q.workspace_size("lsq_linear_bwd", 512, 512, 512, 1, 0)


def test_binding_refuses_host_tensors_and_bad_options():
    x, w, scale, bias = R.layer(4, 8, 64)
    with pytest.raises(ValueError, match="device tensor"):
        w4q.lsq_linear_fwd(x, w, scale)
    with pytest.raises(ValueError, match="device tensor"):
        w4q.lsq_linear_bwd(x, w.to(torch.bfloat16), x)
    with pytest.raises(ValueError, match="device tensor"):
        w4q.w4a16_linear(x, torch.zeros(8, 32, dtype=torch.uint8), scale.half())
    with pytest.raises(ValueError, match="device tensor"):
        w4q.newton_schulz(w)
    with pytest.raises(ValueError, match="device tensor"):
        w4q.muon_step(w, w, w, lr=0.1)
    with pytest.raises(TypeError):
        w4q.newton_schulz(w.double())
    with pytest.raises(TypeError):
        w4q.newton_schulz([1.0])


# ----------------------------------------------------------------- the references themselves
@pytest.mark.parametrize("act", R.ACTS)
def test_reference_gradients_against_differences(act):
    g = R.gen(1)
    x, w, b = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 6), (7, 6), (7,)))
    gy = torch.randn(5, 7, generator=g, dtype=torch.float64)

    def loss(x, w, b):
        return float((R.act(x @ w.t() + b, act) * gy).sum())
    dz = gy * R.dact(x @ w.t() + b, act)
    want = (dz @ w, dz.t() @ x, dz.sum(0))
    for i, (t, grad) in enumerate(zip((x, w, b), want)):
        for j in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[j] = 1e-6
            args = [x, w, b]
            args[i] = t + d.view(t.shape)
            up = loss(*args)
            args[i] = t - d.view(t.shape)
            # fourth-order rest of the difference and the sum's cancellation
            assert abs((up - loss(*args)) / 2e-6 - float(grad.reshape(-1)[j])) < 1e-7
    if act in ("gelu", "silu"):
        z = torch.linspace(-12, 12, 200001, dtype=torch.float64)
        assert float(R.dact(z, act).abs().max()) < R.DACT_MAX


def test_reference_newton_schulz_against_singular_values():
    for r, c in ((5, 9), (9, 5), (6, 6)):
        g = torch.randn(r, c, generator=R.gen(r), dtype=torch.float64)
        u, s, vt = torch.linalg.svd(g, full_matrices=False)
        s = s / (s.norm() + 1e-7)
        for _ in range(5):
            s = R.NS[0] * s + R.NS[1] * s ** 3 + R.NS[2] * s ** 5
        got, _ = R.newton_schulz(g)
        assert torch.allclose(got, u @ torch.diag(s) @ vt, atol=1e-12)
