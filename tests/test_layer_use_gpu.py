"""The layer's operators as a program uses them: sizes that reach the large tiles and split sums, views
at odd addresses, side streams, captured graphs, the whole chain of a training step.  References and
bounds are layer_ref.py's, in 64 bits on the device for the large sizes."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")
from w4a16_group_wise_amd._lib import W4QError  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def within(got, ref, bound, what):
    err = (got.detach().double() - ref).abs()
    ok = err <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} out of bounds, worst {float((err / bound).max()):.3g} of it"


def layer(m, n, k, dev, seed=0):
    return tuple(t.to(dev) for t in R.layer(m, n, k, seed=seed))


def odd(t, by=1):
    """The same values at an address `by` elements past a 256-byte boundary."""
    buf = torch.empty(t.numel() + by + 64, dtype=t.dtype, device=t.device)
    v = buf[by:by + t.numel()].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------------------- large sizes
@pytest.mark.parametrize("m,n,k,act", [(4608, 4352, 2048, "silu"), (3000, 2602, 544, "gelu"), (2304, 5121, 1056, "relu"),
                                       (8200, 2048, 320, "none")])
def test_large_forward_and_backward(dev, m, n, k, act):
    x, w, scale, bias = layer(m, n, k, dev, seed=1)
    res = torch.randn(m, n, generator=R.gen(2, dev), device=dev).to(BF)
    y, w_hat, z = w4q.lsq_linear_fwd(x, w, scale, bias=bias, act=act, residual=res, with_z=True)
    zr, yr, ez, ey = R.linear_fwd(x, w_hat, bias, act, res)
    within(y, yr, R.stored(ey, yr, BF), "y")
    within(z, zr, R.stored(ez, zr, BF), "z")
    del zr, yr, ez, ey
    gy = 1e-3 * torch.randn(m, n, generator=R.gen(3, dev), device=dev)
    gy = gy.to(BF) if act != "gelu" else gy
    gx, gw, gb = w4q.lsq_linear_bwd(x, w_hat, gy, act=act, z=z, with_bias=True)
    _, dx, dw, db, ex, ew, eb = R.linear_bwd(x, w_hat, gy, z, act)
    within(gx, dx, R.stored(ex, dx, BF), "grad_x")
    within(gw, dw, R.stored(ew, dw, F32), "grad_w_hat")
    within(gb, db, R.stored(eb, db, F32), "grad_bias")


@pytest.mark.parametrize("m,n,k", [(1, 4096, 12288), (2, 12288, 512), (16, 9000, 256), (11, 1024, 8192), (40, 12288, 1536), (65, 12288, 1536), (700, 2050, 1024),
                                   (1600, 4096, 4096), (1537, 8200, 2304)])
@pytest.mark.parametrize("dq", [False, True])
def test_large_deployed_layer(dev, m, n, k, dq):
    x, w, scale, bias = layer(m, n, k, dev, seed=4)
    packed, s16 = w4q.quant_pack(w, scale)
    y = w4q.w4a16_linear(x, packed, s16, bias=bias, act="silu", dequant_bf16=dq, out_dtype=F32)
    wr = R.codes(w, scale) * s16.double().repeat_interleave(32, dim=1)
    wr = wr.float().to(BF).double() if dq else wr
    _, yr, _, ey = R.linear_fwd(x, wr, bias, "silu", None)
    ey = ey + R.DACT_MAX * (k + 64) * R.H32 * (x.double().abs() @ wr.abs().t())
    within(y, yr, R.stored(ey, yr, F32), "y")


@pytest.mark.parametrize("b,r,c", [(1, 2048, 2100), (2, 2304, 1300), (1, 1100, 4500), (4, 770, 1024), (1, 64, 70000),
                                   (1, 70000, 33), (3, 48, 300), (3, 300, 49), (2, 65, 65), (70, 32, 32), (4, 39, 5398),
                                   (300, 130, 70)])
def test_large_newton_schulz(dev, b, r, c):
    g = R.gradient(R.gen(b + c, dev), b, r, c, device=dev)
    ref, err = R.newton_schulz(g)
    o = w4q.newton_schulz(g)
    d = torch.linalg.vector_norm(o.double() - ref, dim=(-2, -1))
    assert bool((d <= err).all()), (d / err).max()


@pytest.mark.parametrize("shape", [(40, 200), (200, 64), (100, 300), (1, 70)])
def test_many_steps_on_a_matrix_without_full_rank(dev, shape):
    # what roundings leave where singular values are zero must not grow past the others.  The cubic step
    # s (3 - s^2) / 2 takes every singular value to 1 and none above it
    r, c = shape
    u, v = (torch.randn(k, generator=R.gen(k), dtype=torch.float64) for k in shape)
    u, v = u / u.norm(), v / v.norm()
    g = (u[:, None] * v[None, :]).float().to(dev)
    for steps in (10, 24, 64):
        o = w4q.newton_schulz(g, steps=steps, coeffs=(1.5, -0.5, 0.0)).cpu().double()
        assert float(torch.linalg.matrix_norm(o, 2)) < 1 + 1e-4
        assert abs(float(u @ o @ v) - 1) < 1e-4
        # the published coefficients' bound on any singular value
        o = w4q.newton_schulz(g, steps=steps).cpu().double()
        assert float(torch.linalg.matrix_norm(o, 2)) < 1.21 + 1e-3


@pytest.mark.parametrize("b,r,c", [(2, 1, 1), (1, 1, 40), (1, 40, 1), (3, 5, 33), (2, 64, 31), (1, 48, 5000)])
def test_many_steps_on_short_sides(dev, b, r, c):
    g = torch.randn(b, r, c, generator=R.gen(r), dtype=torch.float64)
    u, _, vh = torch.linalg.svd(g, full_matrices=False)
    o = w4q.newton_schulz(g.float().to(dev), steps=40, coeffs=(1.5, -0.5, 0.0)).cpu().double()
    # The limit is the polar factor.  A step's products (weights 1.5 + 0.5) are off by 2 u, u = 2^-22 for the
    # operands and sqrt(3 k) 2^-23 for the sums (layer_ref.py): while the smallest singular value grows to 1
    # such errors grow with it (norm over smallest singular value); later they add up, one a step, in the
    # directions that turn the factor
    steps = 40
    s = torch.linalg.svdvals(g)
    cond = float((s.norm(dim=1) / s[:, -1]).max())
    unit = 2.0 ** -22 + math.sqrt(3 * max(r, c)) * 2.0 ** -23
    bound = 2 * 2 * unit * (cond + steps) * math.sqrt(min(r, c))
    assert float(torch.linalg.vector_norm(o - u @ vh, dim=(-2, -1)).max()) <= bound


def test_special_values_stay_in_their_matrix_row_or_column(dev):
    g = R.gradient(R.gen(5, dev), 3, 100, 140, device=dev)
    want = w4q.newton_schulz(g)
    for bad in (float("nan"), float("inf")):
        t = g.clone()
        t[0, 99, 139] = bad
        t[2, 0, 0] = bad
        o = w4q.newton_schulz(t)
        assert torch.equal(o[1], want[1]) and bool(torch.isnan(o[0]).all()) and bool(torch.isnan(o[2]).all())
    # lengths of the sums that end inside a stage: a neighbour's infinity is not read as its own zeros
    for k, n in ((96, 90), (160, 66), (544, 300)):
        x, w, scale, bias = layer(70, n, k, dev, seed=k)
        w_hat = w4q.lsq_fwd(w, scale).to(BF)
        gy = torch.randn(70, n, generator=R.gen(1, dev), device=dev).to(BF)
        z = torch.randn(70, n, generator=R.gen(2, dev), device=dev).to(BF)
        y0 = w4q.lsq_linear_fwd(x, None, None, w_hat=w_hat, bias=bias, act="silu")[0]
        packed, s16 = w4q.quant_pack(w, scale)
        p0 = w4q.w4a16_linear(x, packed, s16, bias=bias)
        xb = x.clone()
        xb[7, 3] = float("inf")
        xb[69, k - 1] = float("nan")
        keep = torch.ones(70, dtype=torch.bool, device=dev)
        keep[7] = keep[69] = False
        y = w4q.lsq_linear_fwd(xb, None, None, w_hat=w_hat, bias=bias, act="silu")[0]
        assert torch.equal(y[keep], y0[keep]) and bool(torch.isnan(y[69]).all())
        p = w4q.w4a16_linear(xb, packed, s16, bias=bias)
        assert torch.equal(p[keep], p0[keep]) and bool(torch.isnan(p[69]).all())
        for act in ("none", "gelu"):
            kw = dict(act=act, z=z if act != "none" else None)
            gx0, gw0, _ = w4q.lsq_linear_bwd(x, w_hat, gy, **kw)
            _, gw, _ = w4q.lsq_linear_bwd(xb, w_hat, gy, **kw)
            cols = torch.ones(k, dtype=torch.bool, device=dev)
            cols[3] = cols[k - 1] = False
            assert torch.equal(gw[:, cols], gw0[:, cols]) and bool(torch.isnan(gw[:, k - 1]).all())
            wb = w_hat.clone()
            wb[n - 1, 5] = float("nan")
            gx, _, _ = w4q.lsq_linear_bwd(x, wb, gy, **kw)
            cols = torch.ones(k, dtype=torch.bool, device=dev)
            cols[5] = False
            assert torch.equal(gx[:, cols], gx0[:, cols]) and bool(torch.isnan(gx[:, 5]).all())


def test_offsets_past_32_bits(dev):
    # 2^32 outputs and more: the first and the last rows, and the last matrix of a batch
    m, n, k = 1 << 20, 4096 + 32, 32
    x, w, scale, bias = layer(8, n, k, dev, seed=2)
    x = x.repeat(m // 8, 1)
    ends = torch.cat((torch.arange(100, device=dev), torch.arange(m - 100, m, device=dev)))
    x[ends] = torch.randn(200, k, generator=R.gen(1, dev), device=dev).to(BF)
    y, w_hat, z = w4q.lsq_linear_fwd(x, w, scale, bias=bias, act="silu", with_z=True)
    zr, yr, ez, ey = R.linear_fwd(x[ends], w_hat, bias, "silu", None)
    within(y[ends], yr, R.stored(ey, yr, BF), "y")
    within(z[ends], zr, R.stored(ez, zr, BF), "z")
    packed, s16 = w4q.quant_pack(w, scale)
    res = y[ends]
    out = w4q.w4a16_linear(x, packed, s16, bias=bias, act="silu", residual=y, out_dtype=BF, out=y)
    wr = R.codes(w, scale) * s16.double().repeat_interleave(32, dim=1)
    _, yr, _, ey = R.linear_fwd(x[ends], wr, bias, "silu", res)
    ey = ey + R.DACT_MAX * (k + 64) * R.H32 * (x[ends].double().abs() @ wr.abs().t())
    within(out[ends], yr, R.stored(ey, yr, BF), "deployed")
    del out
    # gradients whose other rows are zero are those of the ends alone
    gy = y.zero_()
    gy[ends] = torch.randn(200, n, generator=R.gen(3, dev), device=dev).to(BF)
    gx, gw, gb = w4q.lsq_linear_bwd(x, w_hat, gy, act="silu", z=z, with_bias=True)
    _, dx, dw, db, ex, ew, eb = R.linear_bwd(x[ends], w_hat, gy[ends], z[ends], "silu")
    within(gx[ends], dx, R.stored(ex, dx, BF), "grad_x")
    within(gw, dw, R.stored(ew, dw, F32), "grad_w_hat")
    within(gb, db, R.stored(eb, db, F32), "grad_bias")
    assert bool((gx[100:m - 100] == 0).all())
    del x, y, z, gy, gx
    b, r, c = 600, 1500, 5000
    g = torch.zeros(b, r, c, device=dev)
    g[0], g[b - 1] = (R.gradient(R.gen(i, dev), r, c, device=dev) for i in (1, 2))
    o = w4q.newton_schulz(g, out=g)
    for i, seed in ((0, 1), (b - 1, 2)):
        ref, err = R.newton_schulz(R.gradient(R.gen(seed, dev), r, c, device=dev))
        assert float(torch.linalg.vector_norm(o[i].double() - ref)) <= float(err)
    assert bool((o[1:b - 1] == 0).all())
    del g, o
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------------- addresses
def test_element_aligned_views(dev):
    # what the interface lets begin at any element gives the bits of the aligned call
    m, n, k = 150, 203, 288
    x, w, scale, bias = layer(m, n, k, dev, seed=6)
    for dtype in (BF, F32):
        res = torch.randn(m, n, generator=R.gen(1, dev), device=dev).to(dtype)
        y, w_hat, z = w4q.lsq_linear_fwd(x, w, scale, bias=bias, act="gelu", residual=res, with_z=True, out_dtype=dtype)
        for by in (1, 3):
            out = odd(torch.zeros(m, n, dtype=dtype, device=dev), by)
            got, _, z2 = w4q.lsq_linear_fwd(x, w, odd(scale, by), bias=odd(bias, by), act="gelu", residual=odd(res, by),
                                            with_z=True, out_dtype=dtype, out=out)
            assert torch.equal(got, y) and torch.equal(z2, z)
            s16 = scale.half()
            packed, _ = w4q.quant_pack(w, scale)
            for rows in (1, 9, m):
                want = w4q.w4a16_linear(x[:rows], packed, s16, bias=bias, act="silu", residual=res[:rows], out_dtype=dtype)
                out = odd(torch.zeros(rows, n, dtype=dtype, device=dev), by)
                got = w4q.w4a16_linear(x[:rows], packed, odd(s16, by), bias=odd(bias, by), act="silu",
                                       residual=odd(res[:rows], by), out_dtype=dtype, out=out)
                assert torch.equal(got, want)
    gy = torch.randn(m, n, generator=R.gen(2, dev), device=dev).to(BF)
    assert all(torch.equal(a, b) for a, b in zip(w4q.lsq_linear_bwd(x, w_hat, gy, act="silu", z=odd(z), with_bias=True),
                                                 w4q.lsq_linear_bwd(x, w_hat, gy, act="silu", z=z, with_bias=True)))
    # (the sum of squares is taken in another order, so not to the bit)
    for shape in ((2, 40, 130), (2, 130, 152)):
        g = R.gradient(R.gen(3, dev), *shape, device=dev)
        for t in (g, g.to(BF)):
            ref, err = R.newton_schulz(t)
            o = w4q.newton_schulz(odd(t), out=odd(torch.zeros_like(t), 3), out_dtype=t.dtype).double()
            slack = R.HB * torch.linalg.vector_norm(ref, dim=(-2, -1)) if t.dtype == BF else 0.0
            assert bool((torch.linalg.vector_norm(o - ref, dim=(-2, -1)) <= err + slack).all())
        w = torch.randn(shape, generator=R.gen(4, dev), device=dev)
        wv, mv = odd(w), odd(torch.zeros_like(g))
        w4q.muon_step(wv, odd(g), mv, lr=0.125, momentum=0.5)  # u = g + m / 2 = 1.5 g
        ref, err = R.newton_schulz(1.5 * g.double())
        sc = math.sqrt(max(1.0, shape[1] / shape[2]))
        assert torch.equal(mv, g)
        within(wv, w.double() - 0.125 * sc * ref, 0.125 * sc * ((err + 3.9 ** 5 * 2 * R.H32)[:, None, None] + 4 * R.H32 * ref.abs())
               + 4 * R.H32 * w.double().abs(), "w")


# --------------------------------------------------------------------- every operator as a call
def calls(dev, m=300, n=520, k=544, seed=0):
    """name -> (inputs, call(inputs, workspace) -> outputs, workspace bytes).  In-place operators get
    copies of what they change."""
    x, w, scale, bias = layer(m, n, k, dev, seed=seed)
    w_hat = w4q.lsq_fwd(w, scale).to(BF)
    gen = R.gen(seed + 1, dev)
    z = torch.randn(m, n, generator=gen, device=dev).to(BF)
    gy = torch.randn(m, n, generator=gen, device=dev).to(BF)
    packed, s16 = w4q.quant_pack(w, scale)
    g = R.gradient(gen, 2, n, k, device=dev)
    thin = R.gradient(gen, 3, 40, k, device=dev)
    size = w4q.workspace_size

    def muon(t, ws):
        w, mom = t[0].clone(), t[2].clone()
        w4q.muon_step(w, t[1], mom, lr=0.02, weight_decay=0.1, workspace=ws)
        return w, mom

    return {
        "forward": ((x, w, scale, bias), lambda t, ws: w4q.lsq_linear_fwd(t[0], t[1], t[2], bias=t[3], act="gelu", with_z=True,
                                                                          workspace=ws), size("lsq_linear_fwd", m, n, k)),
        "backward": ((x, w_hat, gy, z), lambda t, ws: w4q.lsq_linear_bwd(t[0], t[1], t[2], act="silu", z=t[3], with_bias=True,
                                                                        workspace=ws), size("lsq_linear_bwd", m, n, k, 1, 3)),
        "backward of the product": ((x, w_hat, gy), lambda t, ws: w4q.lsq_linear_bwd(t[0], t[1], t[2], with_bias=True,
                                                                                     workspace=ws),
                                    size("lsq_linear_bwd", m, n, k, 1, 0)),
        "deployed": ((x, packed, s16, bias), lambda t, ws: (w4q.w4a16_linear(t[0], t[1], t[2], bias=t[3], act="relu",
                                                                             workspace=ws),), size("w4a16_linear", m, n, k, 0)),
        "deployed, one token": ((x[:1].contiguous(), packed, s16, bias),
                                lambda t, ws: (w4q.w4a16_linear(t[0], t[1], t[2], bias=t[3], act="silu", workspace=ws),),
                                size("w4a16_linear", 1, n, k, 0)),
        "newton_schulz": ((g,), lambda t, ws: (w4q.newton_schulz(t[0], workspace=ws),), size("newton_schulz", 2, n, k)),
        "newton_schulz, thin": ((thin,), lambda t, ws: (w4q.newton_schulz(t[0], workspace=ws),), size("newton_schulz", 3, 40, k)),
        "muon_step": ((g * 3, g, 0.5 * g), muon, size("newton_schulz", 2, n, k)),
    }


NAMES = ["forward", "backward", "backward of the product", "deployed", "deployed, one token", "newton_schulz",
         "newton_schulz, thin", "muon_step"]


def same(a, b):
    return all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_side_streams_and_repeats(dev, name):
    # two streams at once, each call with scratch of its own; twice the same call, the same bits
    inputs, call, _ = calls(dev)[name]
    want = call(inputs, None)
    assert same(call(inputs, None), want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for rep in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(call(inputs, None))
    torch.cuda.synchronize()
    assert all(same(o, want) for per in outs for o in per)


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(dev, name):
    # two graphs with one workspace between them, replayed in turn among eager calls, on new inputs
    inputs, call, bytes_ = calls(dev)[name]
    other, _, _ = calls(dev, seed=9)[name]
    ws = torch.empty(max(bytes_, 1), dtype=torch.uint8, device=dev)
    static = tuple(t.clone() for t in inputs)
    call(static, ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(static, ws))
        graphs.append(g)
    for rep in range(4):
        src = other if rep % 2 else inputs
        for s, t in zip(static, src):
            s.copy_(t)
        want = call(src, None)
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        assert same(outs[rep % 2], want), f"replay {rep}"
        call(other, ws)
        graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        assert same(outs[1 - rep % 2], want), f"replay {rep}, second graph"


# ---------------------------------------------------------------------------------- gradients
@pytest.mark.parametrize("act", R.ACTS)
def test_gradients_against_differences(dev, act):
    """Central differences of L = sum gy * y through the forward's own fp32 outputs.

    With step h on bias[n] or on w_hat[n][k] (dz = h, or h x): the difference's own error is at most
    h^2 / 6 max|act'''| |gy| |dz/dh|^3 summed over the rows (max|act'''| < 0.9), y's error divided by h,
    and the gradient sees z rounded to bf16: |act''| <= 0.8 times 2^-8 |z|.  relu: rows whose z the step
    can carry across 0 are given a zero gy."""
    m, n, k = 40, 24, 64
    x, w, scale, bias = layer(m, n, k, dev, seed=5)
    w_hat = w4q.lsq_fwd(w, scale).to(BF)
    # entries that take the step exactly
    h = 2.0 ** -6
    w_hat[:, 3] = (torch.arange(n, device=dev) - 9).to(BF) / 64
    b = bias

    def fwd(w_hat, b):
        return w4q.lsq_linear_fwd(x, None, None, w_hat=w_hat, bias=b, act=act, with_z=True, out_dtype=F32)
    y, _, z = fwd(w_hat, b)
    gy = torch.randn(m, n, generator=R.gen(3, dev), device=dev)
    if act == "relu":
        gy = torch.where(z.float().abs() > 2 * h * (1 + x[:, 3:4].float().abs()) + 2 ** -6 * z.float().abs(), gy, 0 * gy)
    gx, gw, gb = w4q.lsq_linear_bwd(x, w_hat, gy, act=act, z=z, with_bias=True)
    curved = 0.0 if act in ("none", "relu") else 1.0
    _, _, _, ey = R.linear_fwd(x, w_hat, b, act, None)
    _, _, dw, db, _, ew, eb = R.linear_bwd(x, w_hat, gy, z, act)
    a = gy.double().abs()
    zz = z.double().abs()
    for what, grad, eg, dzdh, step in (
            ("bias", gb.double(), eb, torch.ones(m, 1, dtype=torch.float64, device=dev), lambda s: fwd(w_hat, b + s * h)),
            ("w_hat", gw[:, 3].double(), ew[:, 3], x[:, 3:4].double(),
             lambda s: fwd(torch.cat((w_hat[:, :3], (w_hat[:, 3:4].float() + s * h).to(BF), w_hat[:, 4:]), 1).contiguous(), b))):
        up, dn = step(1.0)[0].double(), step(-1.0)[0].double()
        diff = ((up - dn) * gy.double()).sum(0) / (2 * h)
        d = dzdh.abs()
        bound = (a * (curved * (0.9 * h * h / 6 * d ** 3 + 0.8 * (R.HB * zz) * d) + (ey + R.H32 * (y.double().abs() + 1)) * 2 / h)).sum(0)
        # b + h itself is rounded to fp32
        bound = bound + a.sum(0) * R.H32 * 2 / h + 2 * eg + R.H32 * grad.abs()
        within(diff, grad, bound, what)


# --------------------------------------------------------------------------------- the chain
def test_one_training_step_and_deployment(dev):
    """Two linears with a residual, forward and backward, the LSQ gradients, the Muon step on both,
    packing and the deployed forward; each stage against 64 bits on that stage's own inputs."""
    m, d, hidden = 200, 160, 416
    w1, w2 = (0.05 * torch.randn(s, generator=R.gen(i), dtype=F32).to(dev) for i, s in enumerate(((hidden, d), (d, hidden))))
    s1, s2 = ((0.8 * w.view(w.shape[0], -1, 32).abs().amax(2) / 7).half().float().contiguous() for w in (w1, w2))
    b1 = 0.1 * torch.randn(hidden, generator=R.gen(4)).to(dev)
    x = torch.randn(m, d, generator=R.gen(5)).to(BF).to(dev)
    gy = (1e-2 * torch.randn(m, d, generator=R.gen(6))).to(BF).to(dev)

    h, wh1, z1 = w4q.lsq_linear_fwd(x, w1, s1, bias=b1, act="silu", with_z=True)
    zr, yr, ez, ey = R.linear_fwd(x, R.fake_quant_bf16(w1, s1), b1, "silu", None)
    within(h, yr, R.stored(ey, yr, BF), "hidden")
    y, wh2, _ = w4q.lsq_linear_fwd(h, w2, s2, residual=x)
    _, yr, _, ey = R.linear_fwd(h, R.fake_quant_bf16(w2, s2), None, "none", x)
    within(y, yr, R.stored(ey, yr, BF), "y")

    gh, gw2, _ = w4q.lsq_linear_bwd(h, wh2, gy)
    _, dx, dw, _, ex, ew, _ = R.linear_bwd(h, wh2, gy, None, "none")
    within(gh, dx, R.stored(ex, dx, BF), "grad hidden")
    within(gw2, dw, R.stored(ew, dw, F32), "grad w2")
    gx, gw1, gb1 = w4q.lsq_linear_bwd(x, wh1, gh, act="silu", z=z1, with_bias=True)
    _, dx, dw, db, ex, ew, eb = R.linear_bwd(x, wh1, gh, z1, "silu")
    within(gx, dx, R.stored(ex, dx, BF), "grad x")
    within(gw1, dw, R.stored(ew, dw, F32), "grad w1")
    within(gb1, db, R.stored(eb, db, F32), "grad b1")

    for w, s, gw in ((w1, s1, gw1), (w2, s2, gw2)):
        g, gs, _ = w4q.lsq_bwd(w, s, gw, 1.0 / math.sqrt(32 * 7))
        # the mask on fp32 values: products of a step by 8 and 7 in 64 bits are exact
        delta = s.double().repeat_interleave(32, dim=1)
        inside = (w.double() >= -8 * delta) & (w.double() <= 7 * delta)
        assert torch.equal(g, torch.where(inside, gw, torch.zeros_like(gw)))
        mom, before = torch.zeros_like(w), w.clone()
        w4q.muon_step(w, g, mom, lr=0.02, momentum=0.9)
        assert torch.equal(mom, g)  # 0.9 * 0 + g
        u = g.double() * (1 + float(torch.tensor(0.9)))
        o, err = R.newton_schulz(u)
        sc = math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
        lr = float(torch.tensor(0.02))
        # one rounding of u (2^-24 relative, through five steps of derivative below 3.9), the update's, w's own
        bound = lr * sc * (err + 3.9 ** 5 * 2 * R.H32 + 4 * R.H32 * o.abs()) + 4 * R.H32 * before.double().abs()
        within(w, before.double() - lr * sc * o, bound, "w")

    p1, h1 = w4q.quant_pack(w1, s1)
    p2, h2 = w4q.quant_pack(w2, s2)
    for rows in (1, 6, m):
        hid = w4q.w4a16_linear(x[:rows], p1, h1, bias=b1, act="silu", out_dtype=BF)
        out = w4q.w4a16_linear(hid, p2, h2, residual=x[:rows], out_dtype=BF)
        for got, t, w, s, b, a, r, k in ((hid, x[:rows], w1, h1, b1, "silu", None, d), (out, hid, w2, h2, None, "none", x[:rows], hidden)):
            wr = R.codes(w, s.float()) * s.double().repeat_interleave(32, dim=1)
            _, yr, _, ey = R.linear_fwd(t, wr, b, a, r)
            ey = ey + R.DACT_MAX * (k + 64) * R.H32 * (t.double().abs() @ wr.abs().t())
            within(got, yr, R.stored(ey, yr, BF), f"deployed {rows}")


def test_binding_refuses_overlaps_and_wrong_shapes(dev):
    m, n, k = 16, 64, 64
    x, w, scale, bias = layer(m, n, k, dev)
    packed, s16 = w4q.quant_pack(w, scale)
    buf = torch.zeros(m * n + 64, dtype=BF, device=dev)
    y, shifted = buf[:m * n].view(m, n), buf[8:8 + m * n].view(m, n)
    for call in (lambda **kw: w4q.lsq_linear_fwd(x, w, scale, **kw), lambda **kw: w4q.w4a16_linear(x, packed, s16, out_dtype=BF, **kw)):
        with pytest.raises(ValueError, match="overlap"):
            call(residual=shifted, out=y)
        with pytest.raises(ValueError, match="overlap"):
            call(out=x)
        with pytest.raises(ValueError, match="shape"):
            call(residual=y[:8])
        with pytest.raises(ValueError, match="shape"):
            call(bias=bias[:8])
        with pytest.raises(TypeError):
            call(residual=y.float())
        with pytest.raises(ValueError, match="act must be"):
            call(act="tanh")
        with pytest.raises(ValueError, match="contiguous"):
            call(residual=torch.zeros(n, m, dtype=BF, device=dev).t())
        call(residual=y, out=y)
    with pytest.raises(ValueError, match="overlap"):
        w4q.lsq_linear_fwd(x, w, scale, w_hat=w.view(torch.uint8).view(-1)[:2 * n * k].view(BF).view(n, k))
    with pytest.raises(ValueError, match="together"):
        w4q.lsq_linear_fwd(x, w, None)
    with pytest.raises(ValueError, match="needs z"):
        w4q.lsq_linear_bwd(x, w.to(BF), y, act="silu")
    with pytest.raises(ValueError, match="no gradient"):
        w4q.lsq_linear_bwd(x, w.to(BF), y, with_x=False, with_w=False)
    with pytest.raises(ValueError, match="overlap"):
        w4q.muon_step(w, w, torch.zeros_like(w), lr=0.1)
    with pytest.raises(ValueError, match="overlap"):
        w4q.newton_schulz(w[:32], out=w[16:48])
    with pytest.raises(W4QError):
        w4q.newton_schulz(w, steps=0)
    with pytest.raises(W4QError):
        w4q.w4a16_linear(x[:0], packed, s16)
    with pytest.raises(W4QError):
        w4q.lsq_linear_bwd(x, w.to(BF), y, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
