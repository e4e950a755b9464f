"""Workloads of the quantization-aware layer and its optimiser step: what is timed and compared.

Four operators, each in a plain form (elementary torch operations in 32 bits, 64 where a sum or a
border needs it) and through the library's entry points:

  linear_fwd   y = act(x W^T + bias) + residual with W the bf16 fake-quantised weights of (w, scale)
  linear_bwd   its gradients: grad_x, grad_w_hat (fp32, what lsq_bwd takes) and grad_bias
  w4a16        the deployed form of the same layer on packed INT4 codes, from one row upwards
  ns           the orthogonalised update of Newton-Schulz products, alone
  muon         the whole optimiser step around it: momentum, orthogonalised update, decay, in place

run() goes through the library where `own` is true and through the plain form where it is not.
"""
import math

import torch

own = False

GROUP = 32
NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
ACTS = ("none", "relu", "gelu", "silu")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a lone 256x512 linear on 128 calibration rows: a forward where launches are what costs
        dict(name="fwd_256x512_m128", op="linear_fwd", m=128, d_out=256, d_in=512, act="none", bias=True,
             residual=False, z=False, out="bf16"),
        # a packed batch of odd length through a layer of odd width, everything in the epilogue
        dict(name="fwd_2050x1056_m1531", op="linear_fwd", m=1531, d_out=2050, d_in=1056, act="gelu", bias=True,
             residual=True, z=True, out="bf16"),
        # the gate projection of the hidden-4096 decoder in a training step of 8192 tokens
        dict(name="fwd_gate_m8192", op="linear_fwd", m=8192, d_out=12288, d_in=4096, act="silu", bias=False,
             residual=False, z=True, out="bf16"),
        # the gradients of an odd layer on an odd number of rows
        dict(name="bwd_1001x1056_m1531", op="linear_bwd", m=1531, d_out=1001, d_in=1056, act="gelu", bias=True),
        # the gradients of the gate projection in the same training step
        dict(name="bwd_gate_m8192", op="linear_bwd", m=8192, d_out=12288, d_in=4096, act="silu", bias=False),
        # one decoded token through the down projection, added to the residual stream
        dict(name="w4_down_m1", op="w4a16", m=1, d_out=4096, d_in=12288, act="none", bias=False, residual=True,
             dq=False, out="bf16"),
        # 13 sequences decoding together through the gate projection
        dict(name="w4_gate_m13", op="w4a16", m=13, d_out=12288, d_in=4096, act="silu", bias=True, residual=False,
             dq=False, out="bf16"),
        # a prompt of 2048 tokens through the output projection, added to the residual stream
        dict(name="w4_o_m2048", op="w4a16", m=2048, d_out=4096, d_in=4096, act="none", bias=False, residual=True,
             dq=True, out="bf16"),
        # the update of the lone linear: small dependent products, launches count
        dict(name="ns_256x512", op="ns", batch=1, rows=256, cols=512, out="f32"),
        # the 28 key projections of the hidden-1024 decoder orthogonalised in one call
        dict(name="ns_28x1024x1024", op="ns", batch=28, rows=1024, cols=1024, out="f32"),
        # the optimiser step of one 2048x2048 attention projection
        dict(name="muon_2048x2048", op="muon", batch=1, rows=2048, cols=2048, nesterov=True),
        # the optimiser step of the gate projection (tall)
        dict(name="muon_gate", op="muon", batch=1, rows=12288, cols=4096, nesterov=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges: sizes spread over their logarithm, odd ones among them."""
    most = {op: max(work(c)["flops"] for c in listed() if c["op"] == op)
            for op in ("linear_fwd", "linear_bwd", "w4a16", "ns", "muon")}
    op = rng.choice(["linear_fwd", "linear_bwd", "w4a16", "ns", "muon"])
    while True:
        if op in ("linear_fwd", "linear_bwd"):
            c = dict(op=op, m=_logint(rng, 1, 8192), d_out=_logint(rng, 1, 12288),
                     d_in=GROUP * _logint(rng, 1, 384), act=rng.choice(ACTS), bias=rng.random() < 0.5)
            if op == "linear_fwd":
                c.update(residual=rng.random() < 0.5, z=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
        elif op == "w4a16":
            c = dict(op=op, m=_logint(rng, 1, 2048), d_out=_logint(rng, 1, 12288), d_in=GROUP * _logint(rng, 1, 384),
                     act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                     dq=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
            if c["dq"]:  # rows of whole 256-weight blocks in that reading
                c["d_in"] = 256 * max(1, c["d_in"] // 256)
        else:
            c = dict(op=op, batch=_logint(rng, 1, 28), rows=_logint(rng, 1, 12288), cols=_logint(rng, 1, 12288))
            if op == "ns":
                c["out"] = rng.choice(["bf16", "f32"])
            else:
                c["nesterov"] = rng.random() < 0.5
        if work(c)["flops"] <= most[op]:
            return c


def work(case):
    op = case["op"]
    if op in ("ns", "muon"):
        b, n, k = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # X X^T and A A are symmetric: half their products; B X is whole
        flops = b * NS_STEPS * (float(n) * n * k + float(n) ** 3 + 2.0 * n * n * k)
        per = 20 if op == "muon" else 4 + (4 if case["out"] == "f32" else 2)
        return {"bytes": float(per) * b * n * k, "flops": flops}
    m, n, k = case["m"], case["d_out"], case["d_in"]
    if op == "linear_fwd":
        ob = 2 if case["out"] == "bf16" else 4
        nbytes = 4 * n * k + 4 * n * (k // GROUP) + 2 * n * k + 2 * m * k + ob * m * n
        nbytes += 4 * n * case["bias"] + ob * m * n * case["residual"] + 2 * m * n * case["z"]
        return {"bytes": float(nbytes), "flops": 2.0 * m * n * k}
    if op == "linear_bwd":
        nbytes = 2 * n * k + 2 * m * k + 2 * m * n * (1 + (case["act"] != "none")) + 2 * m * k + 4 * n * k
        nbytes += 4 * n * case["bias"]
        return {"bytes": float(nbytes), "flops": 4.0 * m * n * k}
    ob = 2 if case["out"] == "bf16" else 4
    nbytes = n * k // 2 + 2 * n * (k // GROUP) + 2 * m * k + ob * m * n * (1 + case["residual"]) + 4 * n * case["bias"]
    return {"bytes": float(nbytes), "flops": 2.0 * m * n * k}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, n, k):
    """0.02 N(0, 1) with one weight in 200 ten times as large, and each group's step on the fp16 grid: the
    largest weight of the group over 7, times a factor that a search over [0.4, 1] would take."""
    w = 0.02 * _randn(g, n, k)
    w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.005, 10.0 * w, w)
    amax = w.view(n, k // GROUP, GROUP).abs().amax(dim=2)
    alpha = 0.7 + 0.3 * torch.rand(amax.shape, generator=g, device="cuda")
    scale = (alpha * amax / 7.0).to(torch.float16).float()
    return w, scale


def _activations(g, m, k):
    """N(0, 1) with one lognormal factor for each channel."""
    return (_randn(g, m, k) * torch.exp(0.5 * _randn(g, k))).to(torch.bfloat16)


def _gradient(g, b, rows, cols):
    """Gradients of a few strong directions above noise, as a batch of weights sees them."""
    r = min(16, rows, cols)
    return 1e-3 * (torch.matmul(_randn(g, b, rows, r), _randn(g, b, r, cols)) + _randn(g, b, rows, cols))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("ns", "muon"):
        b, r, c = case["batch"], case["rows"], case["cols"]
        s["grad"] = _gradient(g, b, r, c)
        if op == "muon":
            s["w"] = 0.02 * _randn(g, b, r, c)
            s["m"] = 0.5 * _gradient(g, b, r, c)
        return s
    m, n, k = case["m"], case["d_out"], case["d_in"]
    w, scale = _weights(g, n, k)
    s["x"] = _activations(g, m, k)
    s["bias"] = 0.1 * _randn(g, n) if case["bias"] and op != "linear_bwd" else None
    if op == "linear_fwd":
        s["w"], s["scale"] = w, scale
    elif op == "linear_bwd":
        s["w_hat"] = _fake_quant(w, scale)
        s["grad_y"] = (1e-2 * _randn(g, m, n)).to(torch.bfloat16)
        s["z"] = _randn(g, m, n).to(torch.bfloat16) if case["act"] != "none" else None
    else:
        q = _codes(w, scale).to(torch.int32)
        s["packed"] = ((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).to(torch.uint8).contiguous()
        s["scale_f16"] = scale.to(torch.float16)
    if case.get("residual"):
        s["residual"] = _randn(g, m, n).to(DT[case["out"]])
    else:
        s["residual"] = None
    return s


# ------------------------------------------------------------------------------- plain forms
def _codes(w, scale):
    """The nearest code in [-8, 7], ties to the even one; the quotient in 64 bits, where its borders are exact."""
    d = scale.double().repeat_interleave(GROUP, dim=1)
    q = torch.clamp(torch.round(w.double() / torch.where(d > 0, d, torch.ones_like(d))), -8, 7)
    return torch.where(d > 0, q, torch.zeros_like(q))


def _fake_quant(w, scale):
    return (_codes(w, scale).float() * scale.repeat_interleave(GROUP, dim=1)).to(torch.bfloat16)


def _act(z, act):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(z * -math.sqrt(0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _unpack(packed):
    p = packed.to(torch.int32)
    q = torch.stack((p & 15, p >> 4), dim=2).reshape(p.shape[0], -1)
    return torch.where(q > 7, q - 16, q)


def _epilogue(z, s, case):
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return z, y.to(DT[case["out"]])


def _newton_schulz(g):
    a, b, c = NS
    norm = g.double().square().sum(dim=(-2, -1), keepdim=True).sqrt()
    x = (g.double() / (norm + NS_EPS)).float()
    tall = g.shape[-2] > g.shape[-1]
    if tall:
        x = x.mT.contiguous()
    for _ in range(NS_STEPS):
        p = torch.matmul(x, x.mT.contiguous())
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return x.mT.contiguous() if tall else x


MUON = dict(lr=0.02, momentum=0.95, weight_decay=0.01)


def _muon_scale(case):
    return math.sqrt(max(1.0, case["rows"] / case["cols"]))


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _run_own(s, case, op)
    if op == "linear_fwd":
        w_hat = _fake_quant(s["w"], s["scale"])
        z, y = _epilogue(torch.matmul(s["x"].float(), w_hat.float().t()), s, case)
        return {"y": y, "w_hat": w_hat, "z": z.to(torch.bfloat16) if case["z"] else None}
    if op == "linear_bwd":
        dz = s["grad_y"].float()
        if case["act"] != "none":
            dz = dz * _dact(s["z"].float(), case["act"])
        return {"grad_x": torch.matmul(dz, s["w_hat"].float()).to(torch.bfloat16),
                "grad_w_hat": torch.matmul(dz.t(), s["x"].float()),
                "grad_bias": dz.double().sum(dim=0).float() if case["bias"] else None}
    if op == "w4a16":
        w = _unpack(s["packed"]).float() * s["scale_f16"].float().repeat_interleave(GROUP, dim=1)
        if case["dq"]:
            w = w.to(torch.bfloat16).float()
        return {"y": _epilogue(torch.matmul(s["x"].float(), w.t()), s, case)[1]}
    if op == "ns":
        return {"o": _newton_schulz(s["grad"]).to(DT[case["out"]])}
    mu = MUON["momentum"]
    s["m"].mul_(mu).add_(s["grad"])
    u = s["grad"] + mu * s["m"] if case["nesterov"] else s["m"]
    s["w"].sub_(MUON["lr"] * (_muon_scale(case) * _newton_schulz(u) + MUON["weight_decay"] * s["w"]))
    return {"w": s["w"], "m": s["m"]}


def _run_own(s, case, op):
    import w4a16_group_wise_amd as w4q

    if op == "linear_fwd":
        y, w_hat, z = w4q.lsq_linear_fwd(s["x"], s["w"], s["scale"], bias=s["bias"], act=case["act"],
                                         residual=s["residual"], with_z=case["z"], out_dtype=DT[case["out"]])
        return {"y": y, "w_hat": w_hat, "z": z}
    if op == "linear_bwd":
        gx, gw, gb = w4q.lsq_linear_bwd(s["x"], s["w_hat"], s["grad_y"], act=case["act"], z=s["z"],
                                        with_bias=case["bias"])
        return {"grad_x": gx, "grad_w_hat": gw, "grad_bias": gb}
    if op == "w4a16":
        return {"y": w4q.w4a16_linear(s["x"], s["packed"], s["scale_f16"], bias=s["bias"], act=case["act"],
                                      residual=s["residual"], dequant_bf16=case["dq"], out_dtype=DT[case["out"]])}
    if op == "ns":
        return {"o": w4q.newton_schulz(s["grad"], steps=NS_STEPS, coeffs=NS, eps=NS_EPS, out_dtype=DT[case["out"]])}
    w4q.muon_step(s["w"], s["grad"], s["m"], nesterov=case["nesterov"], update_scale=_muon_scale(case),
                  steps=NS_STEPS, coeffs=NS, eps=NS_EPS, **MUON)
    return {"w": s["w"], "m": s["m"]}


# --------------------------------------------------------------------- 64 bits, written apart
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def polar(g):
        """The same odd polynomials, applied from the side of the longer products' other end: X p(X^T X)."""
        v = g.double()
        v = v / (torch.linalg.vector_norm(v, dim=(-2, -1), keepdim=True) + NS_EPS)
        flip = v.shape[-2] < v.shape[-1]
        if flip:
            v = v.transpose(-2, -1).contiguous()
        for _ in range(NS_STEPS):
            t = v.transpose(-2, -1).contiguous() @ v
            eye = torch.eye(t.shape[-1], dtype=t.dtype, device=t.device)
            v = v @ (NS[0] * eye + t @ (NS[1] * eye + NS[2] * t))
        return v.transpose(-2, -1) if flip else v

    if op == "ns":
        return {"o": polar(s["grad"])}
    if op == "muon":
        g, mu = s["grad"].double(), MUON["momentum"]
        m = mu * s["m"].double() + g
        o = polar(mu * m + g if case["nesterov"] else m)
        w = s["w"].double()
        return {"w": w * (1 - MUON["lr"] * MUON["weight_decay"]) - MUON["lr"] * _muon_scale(case) * o, "m": m}

    def phi(v):
        return 0.5 * (1 + torch.special.erf(v / math.sqrt(2.0)))

    x = s["x"].double()
    if op == "linear_bwd":
        dz = s["grad_y"].double()
        if case["act"] != "none":
            z = s["z"].double()
            sg = torch.sigmoid(z)
            dz = dz * {"relu": (z > 0).double(), "silu": sg + z * sg * (1 - sg),
                       "gelu": phi(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)}[case["act"]]
        return {"grad_x": dz @ s["w_hat"].double(), "grad_w_hat": dz.t().contiguous() @ x,
                "grad_bias": dz.sum(0) if case["bias"] else None}
    if op == "linear_fwd":
        n, k = case["d_out"], case["d_in"]
        d = s["scale"].double().view(n, k // GROUP, 1)
        q = (s["w"].double().view(n, k // GROUP, GROUP) / d.clamp_min(1e-300)).round().clamp(-8, 7)
        w = (d * q).view(n, k).float().to(torch.bfloat16).double()  # the weights are bf16 values by definition
    else:
        p = s["packed"].long()
        q = torch.empty((case["d_out"], case["d_in"]), dtype=torch.float64, device=p.device)
        q[:, 0::2] = (((p & 15) + 8) % 16 - 8).double()
        q[:, 1::2] = (((p >> 4) + 8) % 16 - 8).double()
        w = (q.view(case["d_out"], -1, GROUP) * s["scale_f16"].double().unsqueeze(2)).view(case["d_out"], -1)
        if case["dq"]:
            w = w.float().to(torch.bfloat16).double()
    z = x @ w.t().contiguous()
    if s["bias"] is not None:
        z = z + s["bias"].double()
    y = {"none": lambda v: v, "relu": lambda v: v.clamp_min(0), "gelu": lambda v: v * phi(v),
         "silu": lambda v: v * torch.sigmoid(v)}[case["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    if op == "w4a16":
        return {"y": y}
    return {"y": y, "w_hat": w, "z": z if case["z"] else None}
