"""The layer's product with its epilogue, its gradients, its deployed form, the orthogonalised update
and the Muon step on the GPU, against plain 64-bit forms (layer_ref.py holds them and the bounds)."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
BF, F32 = torch.bfloat16, torch.float32


def within(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    err = (got - ref).abs()
    ok = err <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds, worst {float((err / bound).max()):.3g} of it"


def guarded(shape, dtype, dev, fill=7.0):
    """A contiguous tensor inside a larger buffer, and a check that what lies around it is untouched."""
    n = math.prod(shape)
    pad = 512
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device=dev)
    t = buf[pad:pad + n].view(shape)

    def check():
        assert bool((buf[:pad] == fill).all()) and bool((buf[pad + n:] == fill).all()), "written outside the output"
    return t, check


# --------------------------------------------------------------------------- linear forward
FWD = [(1, 1, 32), (1, 64, 96), (3, 5, 32), (17, 33, 160), (64, 64, 64), (65, 130, 320), (129, 257, 512),
       (300, 515, 1056), (700, 1100, 288), (2100, 1300, 96)]


@pytest.mark.parametrize("m,n,k", FWD)
@pytest.mark.parametrize("act", R.ACTS)
def test_linear_fwd(dev, m, n, k, act):
    x, w, scale, bias = R.layer(m, n, k, seed=m + n)
    for dtype, has_bias, has_res in ((BF, True, True), (F32, True, False), (F32, False, True)):
        res = torch.randn(m, n, generator=R.gen(5)).to(dtype) if has_res else None
        b = bias if has_bias else None
        out, check = guarded((m, n), dtype, dev)
        y, w_hat, z = w4q.lsq_linear_fwd(x.to(dev), w.to(dev), scale.to(dev), bias=b.to(dev) if has_bias else None,
                                         act=act, residual=res.to(dev) if has_res else None, with_z=True,
                                         out_dtype=dtype, out=out)
        torch.cuda.synchronize()
        check()
        wr = R.fake_quant_bf16(w, scale)
        assert torch.equal(w_hat.cpu(), wr)
        zr, yr, ez, ey = R.linear_fwd(x, wr, b, act, res)
        within(y, yr, R.stored(ey, yr, dtype), "y")
        within(z, zr, R.stored(ez, zr, BF), "z")


def test_linear_fwd_given_weights_and_residual_in_place(dev):
    x, w, scale, bias = R.layer(77, 96, 256, seed=3)
    wr = R.fake_quant_bf16(w, scale)
    res = torch.randn(77, 96, generator=R.gen(1)).to(BF)
    y = res.to(dev)
    w_hat = wr.to(dev)
    got, same, z = w4q.lsq_linear_fwd(x.to(dev), None, None, w_hat=w_hat, bias=bias.to(dev), act="silu", residual=y, out=y)
    assert got.data_ptr() == y.data_ptr() and same.data_ptr() == w_hat.data_ptr() and z is None
    zr, yr, ez, ey = R.linear_fwd(x, wr, bias, "silu", res)
    within(got, yr, R.stored(ey, yr, BF), "y")
    assert torch.equal(w_hat.cpu(), wr)


def test_linear_fwd_zero_steps_and_special_values(dev):
    # a step of 0 gives zero weights; an infinite or NaN activation reaches its own row only
    x, w, scale, bias = R.layer(40, 50, 64, seed=4)
    scale[3, 1] = 0.0
    x[5, 7] = float("inf")
    x[6, 8] = float("nan")
    y, w_hat, z = w4q.lsq_linear_fwd(x.to(dev), w.to(dev), scale.to(dev), bias=bias.to(dev), act="relu", with_z=True)
    assert torch.equal(w_hat.cpu(), R.fake_quant_bf16(w, scale)) and bool((w_hat[3, 32:] == 0).all())
    fine = torch.ones(40, dtype=torch.bool)
    fine[5] = fine[6] = False
    zr, yr, ez, ey = R.linear_fwd(x[fine], w_hat.cpu(), bias, "relu", None)
    within(y.cpu()[fine], yr, R.stored(ey, yr, BF), "y")
    assert bool(torch.isnan(z[6]).all()) and bool(torch.isnan(y[6]).all())
    want = x[5].double() * w_hat.cpu().double()
    assert torch.equal(torch.isnan(z[5]).cpu(), torch.isnan(want.sum(1)))


@pytest.mark.parametrize("m,n,k", [(128, 256, 512), (300, 1000, 1056), (1000, 512, 4096)])
def test_linear_fwd_scratch(dev, m, n, k):
    # any scratch, none at all included, up to the order of the sums; the same call twice: the same bits
    x, w, scale, bias = (t.to(dev) for t in R.layer(m, n, k, seed=9))
    need = w4q.workspace_size("lsq_linear_fwd", m, n, k)
    args = dict(bias=bias, act="gelu", out_dtype=F32)
    a = w4q.lsq_linear_fwd(x, w, scale, **args)[0]
    b = w4q.lsq_linear_fwd(x, w, scale, workspace=torch.empty(max(need, 1), dtype=torch.uint8, device=dev), **args)[0]
    c = w4q.lsq_linear_fwd(x, w, scale, workspace=torch.empty(0, dtype=torch.uint8, device=dev), **args)[0]
    assert torch.equal(a, b)
    _, yr, _, ey = R.linear_fwd(x.cpu(), R.fake_quant_bf16(w.cpu(), scale.cpu()), bias.cpu(), "gelu", None)
    within(c, yr, R.stored(ey, yr, F32), "without scratch")


# -------------------------------------------------------------------------- linear backward
BWD = [(1, 1, 32), (1, 96, 64), (3, 5, 32), (33, 17, 160), (64, 64, 64), (130, 65, 320), (515, 300, 288), (700, 1100, 96),
       (2100, 96, 544)]


@pytest.mark.parametrize("m,n,k", BWD)
@pytest.mark.parametrize("act", R.ACTS)
def test_linear_bwd(dev, m, n, k, act):
    x, w, scale, _ = R.layer(m, n, k, seed=m + 2 * n)
    w_hat = R.fake_quant_bf16(w, scale)
    z = torch.randn(m, n, generator=R.gen(2)).to(BF) * 2
    for dtype in (BF, F32):
        gy = (1e-3 * torch.randn(m, n, generator=R.gen(7))).to(dtype)
        gx, gw, gb = w4q.lsq_linear_bwd(x.to(dev), w_hat.to(dev), gy.to(dev), act=act,
                                        z=z.to(dev) if act != "none" else None, with_bias=True)
        _, dx, dw, db, ex, ew, eb = R.linear_bwd(x, w_hat, gy, z, act)
        within(gx, dx, R.stored(ex, dx, BF), f"grad_x {dtype}")
        within(gw, dw, R.stored(ew, dw, F32), f"grad_w_hat {dtype}")
        within(gb, db, R.stored(eb, db, F32), f"grad_bias {dtype}")


def test_linear_bwd_parts_and_ranges(dev):
    # each gradient alone equals the joint call's bits; tiny, huge and zero gradients keep their accuracy
    x, w, scale, _ = (t.to(dev) for t in R.layer(150, 70, 128, seed=8))
    w_hat = R.fake_quant_bf16(w.cpu(), scale.cpu()).to(dev)
    z = torch.randn(150, 70, generator=R.gen(3)).to(BF).to(dev)
    base = torch.randn(150, 70, generator=R.gen(4)).to(BF).to(dev)
    for s in (1.0, 2.0 ** -100, 2.0 ** 90, 0.0):
        gy = base * s
        full = w4q.lsq_linear_bwd(x, w_hat, gy, act="gelu", z=z, with_bias=True)
        for i, kw in enumerate((dict(with_w=False), dict(with_x=False), dict(with_x=False, with_w=False, with_bias=True))):
            part = w4q.lsq_linear_bwd(x, w_hat, gy, act="gelu", z=z, **kw)
            assert torch.equal(part[i], full[i]) and all(part[j] is None for j in range(3) if j != i)
        _, dx, dw, db, ex, ew, eb = R.linear_bwd(x.cpu(), w_hat.cpu(), gy.cpu(), z.cpu(), "gelu")
        within(full[0], dx, R.stored(ex, dx, BF), f"grad_x at {s}")
        within(full[1], dw, R.stored(ew, dw, F32), f"grad_w_hat at {s}")
        within(full[2], db, R.stored(eb, db, F32), f"grad_bias at {s}")


@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_bwd_overflowed_gradient_stays_local(dev, act):
    # an infinite and a NaN entry of grad_y reach their own row of grad_x and column of grad_w_hat only
    x, w, scale, _ = R.layer(70, 90, 64, seed=6)
    w_hat = R.fake_quant_bf16(w, scale)
    z = torch.randn(70, 90, generator=R.gen(5)).to(BF)
    gy = (1e-2 * torch.randn(70, 90, generator=R.gen(6))).to(BF)
    gy[3, 4] = float("inf")
    gy[10, 20] = float("nan")
    gx, gw, gb = w4q.lsq_linear_bwd(x.to(dev), w_hat.to(dev), gy.to(dev), act=act, z=z.to(dev), with_bias=True)
    rows = [i for i in range(70) if i not in (3, 10)]
    cols = [i for i in range(90) if i not in (4, 20)]
    clean = gy.clone()
    clean[3, 4] = clean[10, 20] = 0
    _, dx, dw, db, ex, ew, eb = R.linear_bwd(x, w_hat, clean, z, act)
    within(gx.cpu()[rows], dx[rows], R.stored(ex, dx, BF)[rows], "grad_x")
    within(gw.cpu()[cols], dw[cols], R.stored(ew, dw, F32)[cols], "grad_w_hat")
    within(gb.cpu()[cols], db[cols], R.stored(eb, db, F32)[cols], "grad_bias")
    assert not bool(torch.isfinite(gx[3]).any()) and bool(torch.isnan(gx[10]).all())
    assert not bool(torch.isfinite(gw[4]).any()) and bool(torch.isnan(gw[20]).all())
    assert not bool(torch.isfinite(gb[4])) and bool(torch.isnan(gb[20]))


# ------------------------------------------------------------------------------ deployed form
@pytest.mark.parametrize("m", [1, 2, 7, 16, 17, 40, 300])
@pytest.mark.parametrize("n,k", [(1, 32), (5, 96), (33, 256), (130, 2048), (515, 512), (8200, 256)])
def test_w4a16_linear(dev, m, n, k):
    x, w, scale, bias = R.layer(m, n, k, seed=m)
    q = R.codes(w, scale).to(torch.int32)
    packed = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8).contiguous()
    s16 = scale.to(torch.float16)
    exact_w = (q.double() * s16.double().repeat_interleave(32, dim=1))
    for i, act in enumerate(R.ACTS):
        dq = i % 2 == 1 and k % 256 == 0
        dtype = BF if i < 2 else F32
        res = torch.randn(m, n, generator=R.gen(5)).to(dtype) if i != 2 else None
        b = bias if i != 3 else None
        wr = exact_w.float().to(BF).double() if dq else exact_w
        out, check = guarded((m, n), dtype, dev)
        y = w4q.w4a16_linear(x.to(dev), packed.to(dev), s16.to(dev), bias=None if b is None else b.to(dev), act=act,
                             residual=None if res is None else res.to(dev), dequant_bf16=dq, out_dtype=dtype, out=out)
        torch.cuda.synchronize()
        check()
        _, yr, _, ey = R.linear_fwd(x, wr, b, act, res)
        # the scale multiplies a group's sum in fp32 (and split weights take two products each)
        mag = x.double().abs() @ wr.abs().t()
        ey = ey + R.DACT_MAX * (k + 64) * R.H32 * mag
        within(y, yr, R.stored(ey, yr, dtype), f"{act} dq={dq}")


def test_w4a16_linear_without_epilogue_is_the_product(dev):
    # nothing in the epilogue: the bits of w4a16_gemm / w4a16_gemm_dq, at every row count's kernel
    for m, n, k in ((1, 4096, 2048), (9, 300, 512), (16, 8192, 512), (200, 700, 512), (1000, 4200, 288)):
        x, w, scale, _ = (t.to(dev) for t in R.layer(m, n, k, seed=2))
        packed, s16 = w4q.quant_pack(w, scale)
        assert torch.equal(w4q.w4a16_linear(x, packed, s16), w4q.w4a16_gemm(x, packed, s16))
        if k % 256 == 0:
            # (with less scratch than its own fastest schedule asks for, which may be another one)
            less = min(w4q.workspace_size("w4a16_gemm_dq", m, n, k), w4q.workspace_size("w4a16_linear", m, n, k, 1) - 256)
            ws = torch.empty(max(less, 0), dtype=torch.uint8, device=dev)
            want = w4q.w4a16_gemm_dq(x, packed, s16, out_dtype=BF, workspace=ws)
            assert torch.equal(w4q.w4a16_linear(x, packed, s16, dequant_bf16=True, out_dtype=BF, workspace=ws), want)


# ------------------------------------------------------------------------------ Newton-Schulz
NS = [(1, 1, 1), (1, 1, 40), (1, 40, 1), (2, 3, 5), (1, 31, 33), (3, 33, 31), (1, 64, 64), (2, 65, 200), (2, 200, 65),
      (1, 129, 1000), (1, 1000, 129), (1, 512, 520), (5, 256, 300), (1, 1100, 1300), (40, 24, 24), (1, 2304, 1500)]


@pytest.mark.parametrize("b,r,c", NS)
def test_newton_schulz(dev, b, r, c):
    g = R.gradient(R.gen(b + r), b, r, c)
    ref, err = R.newton_schulz(g)
    out, check = guarded((b, r, c), F32, dev)
    o = w4q.newton_schulz(g.to(dev), out=out)
    torch.cuda.synchronize()
    check()
    d = torch.linalg.vector_norm(o.cpu().double() - ref, dim=(-2, -1))
    assert bool((d <= err).all()), (d, err)
    # bf16 in (the reference takes the same values), bf16 out: one more rounding
    gb = g.to(BF)
    refb, errb = R.newton_schulz(gb)
    ob = w4q.newton_schulz(gb.to(dev), out_dtype=BF)
    assert ob.dtype == BF
    d = torch.linalg.vector_norm(ob.cpu().double() - refb, dim=(-2, -1))
    assert bool((d <= errb + R.HB * torch.linalg.vector_norm(refb, dim=(-2, -1))).all())


def test_newton_schulz_options(dev):
    g = R.gradient(R.gen(1), 70, 90)
    for steps in (1, 2, 7):
        ref, err = R.newton_schulz(g, steps=steps)
        o = w4q.newton_schulz(g.to(dev), steps=steps)
        assert o.shape == g.shape and float(torch.linalg.vector_norm(o.cpu().double() - ref)) <= float(err)
    # the convergent cubic iteration has a polar factor as its limit: orthonormal rows
    o = w4q.newton_schulz(torch.randn(40, 200, generator=R.gen(2)).to(dev), steps=40, coeffs=(1.5, -0.5, 0.0)).cpu().double()
    assert float((o @ o.t() - torch.eye(40, dtype=torch.float64)).abs().max()) < 1e-5
    # in place, and scale invariance over the whole range of fp32
    want = w4q.newton_schulz(g.to(dev), eps=0.0)
    for s in (2.0 ** -120, 2.0 ** 120):
        t = (g * s).to(dev)
        got = w4q.newton_schulz(t, eps=0.0, out=t)
        assert got.data_ptr() == t.data_ptr()
        assert torch.allclose(got, want, rtol=1e-4, atol=1e-6)


def test_newton_schulz_zero_and_special_values(dev):
    g = R.gradient(R.gen(3), 3, 50, 60)
    g[1] = 0
    g[2, 4, 5] = float("nan")
    o = w4q.newton_schulz(g.to(dev)).cpu()
    ref, err = R.newton_schulz(g[:1])
    assert float(torch.linalg.vector_norm(o[:1].double() - ref)) <= float(err)
    assert bool((o[1] == 0).all())
    assert bool(torch.isnan(o[2]).all())


@pytest.mark.parametrize("b,r,c,nesterov", [(1, 64, 96, True), (1, 300, 130, False), (3, 33, 70, True), (1, 1, 7, True),
                                            (2, 520, 512, False)])
def test_muon_step(dev, b, r, c, nesterov):
    g = R.gen(r + c)
    w = 0.02 * torch.randn(b, r, c, generator=g)
    m = 0.5 * R.gradient(g, b, r, c)
    wd, md = w.to(dev), m.to(dev)
    lr, mu, decay, scale = 0.02, 0.95, 0.1, math.sqrt(max(1, r / c))
    lr32, mu32, dec32 = (float(torch.tensor(v)) for v in (lr, mu, decay))
    wr, mr = w.double(), m.double()
    ew = torch.zeros_like(wr)
    em = torch.zeros_like(mr)
    for step in range(3):
        grad = R.gradient(g, b, r, c)
        w4q.muon_step(wd, grad.to(dev), md, lr=lr, momentum=mu, nesterov=nesterov, weight_decay=decay)
        em = mu32 * em + R.H32 * (mu32 * mr.abs() + grad.double().abs() + mr.abs())
        mr = mu32 * mr + grad.double()
        u = grad.double() + mu32 * mr if nesterov else mr
        o, err = R.newton_schulz(u)
        # momentum's own error passes through the update's derivative (3.9 per step on U / ||U||)
        rel = torch.linalg.vector_norm(em + R.H32 * u.abs(), dim=(-2, -1)) / torch.linalg.vector_norm(u, dim=(-2, -1))
        eo = (err + 2 * 3.9 ** 5 * rel)[:, None, None]
        ew = ew * (1 + lr32 * dec32) + lr32 * scale * (eo + 4 * R.H32 * o.abs()) + 4 * R.H32 * wr.abs()
        wr = wr - lr32 * (scale * o + dec32 * wr)
        within(md, mr, em + 1e-30, f"m after step {step}")
        within(wd, wr, ew, f"w after step {step}")


def test_matrix_and_batch_forms_agree(dev):
    g = R.gradient(R.gen(4), 3, 100, 140).to(dev)
    batch = w4q.newton_schulz(g)
    ref, err = R.newton_schulz(g.cpu())
    for i in range(3):
        one = w4q.newton_schulz(g[i].contiguous())
        assert one.shape == (100, 140)
        assert float(torch.linalg.vector_norm(one.cpu().double() - ref[i])) <= float(err[i])
    assert bool((torch.linalg.vector_norm(batch.cpu().double() - ref, dim=(-2, -1)) <= err).all())
