"""Cases of the training operators around the optimizer: layer norm, the linear
layer's three products and 8-bit activation checkpoints, each in a plain form
(elementary torch operations in float32) and as a caller of the library runs it.

`own` selects: False computes the plain forms, True calls the library.
"""

import math

import torch

own = False

GROUP = 32          # columns that share one exponent of an 8-bit checkpoint
_GELU_C = math.sqrt(2.0 / math.pi)
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_handles = {}


def _lib():
    """The package and this process's handle (a training program keeps one)."""
    import newton_schulz_matrix_step_amd as nsm
    if "h" not in _handles:
        _handles["h"] = nsm.muon_init(torch.cuda.current_device())
    return nsm, _handles["h"]


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one decoding-sized batch through the norm: launch latency
        {"name": "ln fwd 16x768 bf16", "op": "ln_fwd", "rows": 16, "cols": 768, "dtype": "bf16", "params": "bf16"},
        # a float32 residual stream with an odd number of tokens
        {"name": "ln fwd 8191x2048 f32", "op": "ln_fwd", "rows": 8191, "cols": 2048, "dtype": "f32", "params": "f32"},
        # a large layer's pre-norm in training, its residual gradient added
        {"name": "ln bwd 8192x4096 bf16", "op": "ln_bwd", "rows": 8192, "cols": 4096, "dtype": "bf16",
         "params": "bf16", "add": True},
        # one token through the large layer's up projection: the weight is read once
        {"name": "lin fwd 1 4096-14336", "op": "lin_fwd", "rows": 1, "in": 4096, "out": 14336, "dtype": "bf16",
         "act": "relu_sq", "bias": False, "residual": False, "layout": "in_out"},
        # up projection of the 350M-style model over one batch
        {"name": "lin fwd 8192 1024-4096 gelu", "op": "lin_fwd", "rows": 8192, "in": 1024, "out": 4096,
         "dtype": "bf16", "act": "gelu", "bias": True, "residual": False, "layout": "in_out"},
        # down projection of the large layer with the residual stream added
        {"name": "lin fwd 4096 14336-4096 res", "op": "lin_fwd", "rows": 4096, "in": 14336, "out": 4096,
         "dtype": "bf16", "act": "none", "bias": True, "residual": True, "layout": "out_in"},
        # a small float32 model's projection
        {"name": "lin fwd 300 768-768 f32", "op": "lin_fwd", "rows": 300, "in": 768, "out": 768, "dtype": "f32",
         "act": "gelu", "bias": True, "residual": False, "layout": "in_out"},
        # down projection's input gradient through the activation, from the 8-bit pre-activation (ragged batch)
        {"name": "lin dx 4001 1024-4096 z8", "op": "lin_dx", "rows": 4001, "in": 4096, "out": 1024, "dtype": "bf16",
         "act": "gelu", "z": "act8", "act_out": True, "add": False, "layout": "in_out"},
        # up projection's weight and bias gradient from the 8-bit layer input
        {"name": "lin dw 8192 1024-4096 x8", "op": "lin_dw", "rows": 8192, "in": 1024, "out": 4096, "dtype": "bf16",
         "x": "act8", "db": True, "layout": "in_out", "dw": "bf16"},
        # a large activation to 8 bits and back
        {"name": "act8 16384x4096 bf16", "op": "act8", "rows": 16384, "cols": 4096, "dtype": "bf16"},
        # a small float32 one whose rows end inside a group
        {"name": "act8 777x1000 f32", "op": "act8", "rows": 777, "cols": 1000, "dtype": "f32"},
        # the whole sub-block of one layer, forward and backward, with 8-bit checkpoints
        {"name": "mlp step 4096 1024-4096", "op": "mlp", "rows": 4096, "cols": 1024, "ff": 4096, "dtype": "bf16",
         "act": "gelu", "layout": "in_out"},
    ]


def _logint(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lin_fwd", "lin_fwd", "lin_dx", "lin_dw", "act8", "mlp"])
    dt = "bf16" if rng.random() < 0.75 else "f32"
    if op in ("ln_fwd", "ln_bwd", "act8"):
        step = 1 if rng.random() < 0.2 else 8
        cols = _logint(rng, 64, 8192, step)
        rows = _logint(rng, 1, min(16384, (1 << 26) // cols))
        c = {"op": op, "rows": rows, "cols": cols, "dtype": dt}
        if op != "act8":
            c["params"] = rng.choice([dt, "f32"])
        if op == "ln_bwd":
            c["add"] = rng.random() < 0.5
        return c
    dt = "bf16" if op == "mlp" else dt
    budget = 4.0e11 if dt == "bf16" else 2.0e10
    step = 1 if rng.random() < 0.1 else 8
    nin = _logint(rng, 128, 8192, step)
    nout = _logint(rng, 128, 8192, step)
    if op == "mlp":
        nin, nout = _logint(rng, 128, 2048, 8), _logint(rng, 256, 8192, 8)
        rows = _logint(rng, 16, max(16, min(8192, int(budget / (12.0 * nin * nout)))))
        return {"op": op, "rows": rows, "cols": nin, "ff": nout, "dtype": dt, "act": rng.choice(["gelu", "relu_sq"]),
                "layout": rng.choice(["in_out", "out_in"])}
    rows = _logint(rng, 1 if op == "lin_fwd" else 16, max(16, min(16384, int(budget / (2.0 * nin * nout)))))
    c = {"op": op, "rows": rows, "in": nin, "out": nout, "dtype": dt, "layout": rng.choice(["in_out", "out_in"])}
    if op == "lin_fwd":
        c.update(act=rng.choice(["none", "gelu", "relu_sq"]), bias=rng.random() < 0.7, residual=rng.random() < 0.4)
    elif op == "lin_dx":
        z = rng.choice(["act8", "full", "none"])
        c.update(z=z, act="none" if z == "none" else rng.choice(["gelu", "relu_sq"]),
                 act_out=z != "none" and rng.random() < 0.5, add=rng.random() < 0.3)
    else:
        c.update(x=rng.choice(["act8", "full"]), db=rng.random() < 0.7, dw=rng.choice([dt, "f32"]))
    return c


# ---- inputs ------------------------------------------------------------------

def _pack8(x):
    """8-bit checkpoint of x: int8 codes and one exponent byte per GROUP columns
    of a row; an element is code * 2^(exponent byte - 127)."""
    r, c = x.shape
    g = -(-c // GROUP)
    p = torch.zeros(r, g * GROUP, dtype=torch.float32, device=x.device)
    p[:, :c] = x.float()
    p = p.view(r, g, GROUP)
    m, e = torch.frexp(p.abs().amax(dim=2))
    # smallest power of two with amax / 2^k <= 127, at least 2^-126
    k = (e - 7 + (m > 127.0 / 128.0).to(e.dtype)).clamp_min(-126)
    q = torch.round(torch.ldexp(p, -k.unsqueeze(2)))
    return q.view(r, g * GROUP)[:, :c].to(torch.int8).contiguous(), (k + 127).to(torch.uint8).contiguous()


def _unpack8(q, e):
    r, c = q.shape
    k = (e.to(torch.int32) - 127).repeat_interleave(GROUP, dim=1)[:, :c]
    return torch.ldexp(q.float(), k)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]

    def rnd(*shape, std=1.0, mean=0.0, dtype=dt):
        t = torch.empty(*shape, device=dev, dtype=torch.float32)
        return t.normal_(mean, std, generator=g).to(dtype)

    def out(*shape, dtype=dt):
        return torch.empty(*shape, device=dev, dtype=dtype)

    op = case["op"]
    s = {"case": case}
    rows = case["rows"]
    if op in ("ln_fwd", "ln_bwd"):
        n, pt = case["cols"], _DT[case["params"]]
        # a residual stream: rows of different sizes, a common offset
        s["x"] = (rnd(rows, n, dtype=torch.float32) * rnd(rows, 1, dtype=torch.float32).exp() + 0.3).to(dt)
        s["gain"], s["bias"] = rnd(n, std=0.1, mean=1.0, dtype=pt), rnd(n, std=0.1, dtype=pt)
        if op == "ln_fwd":
            s["y"], s["mean"], s["rstd"] = out(rows, n), out(rows, dtype=torch.float32), out(rows, dtype=torch.float32)
        else:
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = (xf - s["mean"][:, None]).square().mean(1).add(1e-5).rsqrt()
            s["dy"] = rnd(rows, n, std=1e-2)
            s["add"] = rnd(rows, n, std=1e-2) if case["add"] else None
            s["dx"], s["dgain"], s["dbias"] = out(rows, n), out(n, dtype=pt), out(n, dtype=pt)
        return s
    if op == "act8":
        n = case["cols"]
        s["x"] = rnd(rows, n) * rnd(rows, 1).exp()
        s["q"], s["e"] = out(rows, n, dtype=torch.int8), out(rows, -(-n // GROUP), dtype=torch.uint8)
        s["y"] = out(rows, n)
        return s
    if op == "mlp":
        n, f = case["cols"], case["ff"]
        t = case["layout"] == "out_in"
        s["x"], s["dy"] = rnd(rows, n), rnd(rows, n, std=1e-2)
        s["gain"], s["beta"] = rnd(n, std=0.1, mean=1.0), rnd(n, std=0.1)
        s["w1"] = rnd(f, n, std=n ** -0.5) if t else rnd(n, f, std=n ** -0.5)
        s["w2"] = rnd(n, f, std=f ** -0.5) if t else rnd(f, n, std=f ** -0.5)
        s["b1"], s["b2"] = rnd(f, std=0.1), rnd(n, std=0.1)
        s["xn"], s["h"], s["y"] = out(rows, n), out(rows, f), out(rows, n)
        s["mean"], s["rstd"] = out(rows, dtype=torch.float32), out(rows, dtype=torch.float32)
        for k, c in (("xn8", n), ("z8", f)):
            s[k] = (out(rows, c, dtype=torch.int8), out(rows, -(-c // GROUP), dtype=torch.uint8))
        s["dz"], s["h2"], s["dxn"], s["dx"] = out(rows, f), out(rows, f), out(rows, n), out(rows, n)
        s["dw1"], s["dw2"], s["db1"], s["db2"] = out(*s["w1"].shape), out(*s["w2"].shape), out(f), out(n)
        s["dgain"], s["dbeta"] = out(n), out(n)
        return s
    k, n = case["in"], case["out"]
    wshape = (n, k) if case["layout"] == "out_in" else (k, n)
    if op == "lin_fwd":
        s["x"], s["w"] = rnd(rows, k), rnd(*wshape, std=k ** -0.5)
        s["bias"] = rnd(n, std=0.1) if case["bias"] else None
        s["res"] = rnd(rows, n) if case["residual"] else None
        s["y"] = out(rows, n)
    elif op == "lin_dx":
        s["dy"], s["w"] = rnd(rows, n, std=1e-2), rnd(*wshape, std=n ** -0.5)
        s["z"] = None if case["z"] == "none" else rnd(rows, k)
        if case["z"] == "act8":
            s["z"] = _pack8(s["z"])
        s["add"] = rnd(rows, k, std=1e-2) if case["add"] else None
        s["dx"], s["act_out"] = out(rows, k), out(rows, k) if case["act_out"] else None
    else:
        s["x"], s["dy"] = rnd(rows, k), rnd(rows, n, std=1e-2)
        if case["x"] == "act8":
            s["x"] = _pack8(s["x"])
        s["dw"] = out(*wshape, dtype=_DT[case["dw"]])
        s["db"] = out(n) if case["db"] else None
    return s


# ---- plain forms -------------------------------------------------------------

def _act(z, kind):
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(_GELU_C * (z + 0.044715 * z * z * z)))
    if kind == "relu_sq":
        r = z.clamp_min(0.0)
        return r * r
    return z


def _act_grad(z, kind):
    if kind == "gelu":
        t = torch.tanh(_GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _GELU_C * (1.0 + 3 * 0.044715 * z * z)
    if kind == "relu_sq":
        return 2.0 * z.clamp_min(0.0)
    return torch.ones_like(z)


def _ln_plain(x, gain, bias, eps=1e-5):
    xf = x.float()
    mean = xf.mean(1)
    d = xf - mean[:, None]
    rstd = (d * d).mean(1).add(eps).rsqrt()
    return d * rstd[:, None] * gain.float() + bias.float(), mean, rstd


def _ln_grad_plain(dy, x, gain, mean, rstd, add):
    dyf = dy.float()
    xh = (x.float() - mean[:, None]) * rstd[:, None]
    a = dyf * gain.float()
    dx = rstd[:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    if add is not None:
        dx = dx + add.float()
    return dx, (dyf * xh).sum(0), dyf.sum(0)


def _w_in_out(w, layout):
    return w.float().t() if layout == "out_in" else w.float()


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "ln_fwd":
        y, mean, rstd = _ln_plain(s["x"], s["gain"], s["bias"])
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dg, db = _ln_grad_plain(s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], s["add"])
        pt = _DT[case["params"]]
        return {"dx": dx.to(dt), "dgain": dg.to(pt), "dbias": db.to(pt)}
    if op == "act8":
        return {"y": _unpack8(*_pack8(s["x"])).to(dt)}
    lay = case["layout"]
    if op == "lin_fwd":
        z = s["x"].float() @ _w_in_out(s["w"], lay)
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(dt)}
    if op == "lin_dx":
        dx = s["dy"].float() @ _w_in_out(s["w"], lay).t()
        r = {}
        if s["z"] is not None:
            z = _unpack8(*s["z"]) if case["z"] == "act8" else s["z"].float()
            dx = dx * _act_grad(z, case["act"])
            if case["act_out"]:
                r["act_out"] = _act(z, case["act"]).to(dt)
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return {"dx": dx.to(dt), **r}
    if op == "lin_dw":
        x = _unpack8(*s["x"]) if case["x"] == "act8" else s["x"].float()
        dy = s["dy"].float()
        dw = dy.t() @ x if lay == "out_in" else x.t() @ dy
        r = {"dw": dw.to(_DT[case["dw"]])}
        if case["db"]:
            r["db"] = dy.sum(0).to(dt)
        return r
    # mlp: every operator rounds its result once; the backward pass sees the 8-bit checkpoints
    act = case["act"]
    w1, w2 = _w_in_out(s["w1"], lay), _w_in_out(s["w2"], lay)
    xn, mean, rstd = _ln_plain(s["x"], s["gain"], s["beta"])
    xn8, xn = _unpack8(*_pack8(xn)), xn.to(dt).float()
    z = xn @ w1 + s["b1"].float()
    z8, h = _unpack8(*_pack8(z)), _act(z, act).to(dt).float()
    y = h @ w2 + s["b2"].float() + s["x"].float()
    dy = s["dy"].float()
    dz = ((dy @ w2.t()) * _act_grad(z8, act)).to(dt).float()
    h2 = _act(z8, act).to(dt).float()
    dw2, dw1 = h2.t() @ dy, xn8.t() @ dz
    if lay == "out_in":
        dw1, dw2 = dw1.t().contiguous(), dw2.t().contiguous()
    dxn = (dz @ w1.t()).to(dt)
    dx, dg, db = _ln_grad_plain(dxn, s["x"], s["gain"], mean, rstd, s["dy"])
    return {"y": y.to(dt), "dx": dx.to(dt), "dw1": dw1.to(dt), "dw2": dw2.to(dt), "db1": dz.sum(0).to(dt),
            "db2": dy.sum(0).to(dt), "dgain": dg.to(dt), "dbeta": db.to(dt)}


# ---- the library's calls -------------------------------------------------------

def _run_own(s):
    nsm, h = _lib()
    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        nsm.muon_layernorm_forward(h, s["x"], s["gain"], s["bias"], s["y"], mean=s["mean"], rstd=s["rstd"], eps=1e-5)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_bwd":
        nsm.muon_layernorm_backward(h, s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], s["dx"], s["dgain"],
                                    dbias=s["dbias"], add=s["add"])
        return {"dx": s["dx"], "dgain": s["dgain"], "dbias": s["dbias"]}
    if op == "act8":
        a = nsm.Act8(s["q"], s["e"])
        nsm.muon_act_encode(h, s["x"], a)
        nsm.muon_act_decode(h, a, s["y"])
        return {"y": s["y"]}
    lay = case["layout"]
    if op == "lin_fwd":
        nsm.muon_linear_forward(h, s["x"], s["w"], s["y"], bias=s["bias"], act=case["act"], residual=s["res"],
                                w_layout=lay)
        return {"y": s["y"]}
    if op == "lin_dx":
        z = nsm.Act8(*s["z"]) if case["z"] == "act8" else s["z"]
        nsm.muon_linear_grad_input(h, s["dy"], s["w"], s["dx"], act=case["act"], z=z, act_out=s["act_out"],
                                   add=s["add"], w_layout=lay)
        return {"dx": s["dx"], **({"act_out": s["act_out"]} if case["act_out"] else {})}
    if op == "lin_dw":
        x = nsm.Act8(*s["x"]) if case["x"] == "act8" else s["x"]
        nsm.muon_linear_grad_weight(h, x, s["dy"], s["dw"], db=s["db"], w_layout=lay)
        return {"dw": s["dw"], **({"db": s["db"]} if case["db"] else {})}
    act = case["act"]
    xn8, z8 = nsm.Act8(*s["xn8"]), nsm.Act8(*s["z8"])
    nsm.muon_layernorm_forward(h, s["x"], s["gain"], s["beta"], s["xn"], mean=s["mean"], rstd=s["rstd"], eps=1e-5,
                               y8=xn8)
    nsm.muon_linear_forward(h, s["xn"], s["w1"], s["h"], bias=s["b1"], act=act, z_out=z8, w_layout=lay)
    nsm.muon_linear_forward(h, s["h"], s["w2"], s["y"], bias=s["b2"], residual=s["x"], w_layout=lay)
    nsm.muon_linear_grad_input(h, s["dy"], s["w2"], s["dz"], act=act, z=z8, act_out=s["h2"], w_layout=lay)
    nsm.muon_linear_grad_weight(h, s["h2"], s["dy"], s["dw2"], db=s["db2"], w_layout=lay)
    nsm.muon_linear_grad_input(h, s["dz"], s["w1"], s["dxn"], w_layout=lay)
    nsm.muon_linear_grad_weight(h, xn8, s["dz"], s["dw1"], db=s["db1"], w_layout=lay)
    nsm.muon_layernorm_backward(h, s["dxn"], s["x"], s["gain"], s["mean"], s["rstd"], s["dx"], s["dgain"],
                                dbias=s["dbeta"], add=s["dy"])
    return {k: s[k] for k in ("y", "dx", "dw1", "dw2", "db1", "db2", "dgain", "dbeta")}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    r, op = case["rows"], case["op"]
    if op == "ln_fwd":
        n = case["cols"]
        p = 2 if case["params"] == "bf16" else 4
        return {"bytes": 2 * r * n * b + 2 * n * p + 8 * r, "flops": 8 * r * n}
    if op == "ln_bwd":
        n = case["cols"]
        p = 2 if case["params"] == "bf16" else 4
        return {"bytes": (3 + bool(case["add"])) * r * n * b + 3 * n * p + 8 * r, "flops": 14 * r * n}
    if op == "act8":
        # to 8 bits (read, write codes and exponents) and back
        n = case["cols"]
        return {"bytes": 2 * r * n * b + 2 * r * (n + -(-n // GROUP)), "flops": 4 * r * n}
    if op == "mlp":
        n, f = case["cols"], case["ff"]
        e8 = r * (n + -(-n // GROUP)) + r * (f + -(-f // GROUP))
        return {"bytes": b * (4 * r * n + 4 * n * f) + 2 * e8 + 8 * r + b * (2 * f + 6 * n), "flops": 12 * r * n * f}
    k, n = case["in"], case["out"]
    flops = 2 * r * k * n
    if op == "lin_fwd":
        return {"bytes": b * (r * k + k * n + r * n * (1 + case["residual"]) + n * case["bias"]), "flops": flops}
    if op == "lin_dx":
        zb = {"none": 0, "full": b * r * k, "act8": r * (k + -(-k // GROUP))}[case["z"]]
        return {"bytes": b * (r * n + k * n + r * k * (1 + case["add"] + case["act_out"])) + zb, "flops": flops}
    xb = b * r * k if case["x"] == "full" else r * (k + -(-k // GROUP))
    return {"bytes": xb + b * r * n + (2 if case["dw"] == "bf16" else 4) * k * n + b * n * case["db"],
            "flops": flops + r * n * case["db"]}


# ---- the definitions in float64 -------------------------------------------------

def _x_round(v, dt):
    """Rounding to the storage type, from float64."""
    return v.to(dt).double()


def _x_quant(v):
    """v rounded to its 8-bit checkpoint: per group of GROUP columns the step is
    the smallest power of two (not under 2^-126) that keeps every code within 127."""
    n = v.shape[1]
    pad = torch.nn.functional.pad(v, (0, (-n) % GROUP)).unflatten(1, (-1, GROUP))
    top = pad.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2((top / 127.0).clamp_min(2.0 ** -126))))
    step = torch.where(top > 127.0 * step, 2 * step, torch.where(top <= 63.5 * step, step / 2, step))
    step = step.clamp_min(2.0 ** -126)
    return ((pad / step).round() * step).flatten(1)[:, :n]


def _x_decode(pair):
    q, e = pair
    step = torch.exp2(e.double() - 127.0)
    return q.double() * step[:, torch.arange(q.shape[1], device=q.device) // GROUP]


def _x_act(z, kind):
    """(activation, derivative)"""
    if kind == "gelu":
        u = _GELU_C * (z + 0.044715 * z ** 3)
        sig = torch.sigmoid(2 * u)   # (1 + tanh u) / 2
        return z * sig, sig + z * 2 * sig * (1 - sig) * _GELU_C * (1 + 0.134145 * z ** 2)
    if kind == "relu_sq":
        pos = (z > 0).double()
        return z * z * pos, 2 * z * pos
    return z, torch.ones_like(z)


def _x_norm(x, gain, bias):
    var, mean = torch.var_mean(x, dim=1, unbiased=False)
    rstd = 1.0 / torch.sqrt(var + 1e-5)
    return (x - mean[:, None]) * rstd[:, None] * gain + bias, mean, rstd


def _x_norm_grad(dy, x, gain, mean, rstd, add):
    n = x.shape[1]
    xh = (x - mean[:, None]) * rstd[:, None]
    gy = gain * dy
    c1, c2 = gy.sum(1, keepdim=True) / n, (gy * xh).sum(1, keepdim=True) / n
    dx = (gy - c1 - c2 * xh) * rstd[:, None]
    return (dx if add is None else dx + add), torch.einsum("ij,ij->j", dy, xh), torch.einsum("ij->j", dy)


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], _DT[case["dtype"]]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if op == "ln_fwd":
        y, mean, rstd = _x_norm(d["x"], d["gain"], d["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dg, db = _x_norm_grad(d["dy"], d["x"], d["gain"], d["mean"], d["rstd"], d.get("add"))
        return {"dx": dx, "dgain": dg, "dbias": db}
    if op == "act8":
        return {"y": _x_quant(d["x"])}
    flip = case["layout"] == "out_in"
    if op == "lin_fwd":
        z = d["x"] @ (d["w"].t() if flip else d["w"])
        z = z + d["bias"] if "bias" in d else z
        y = _x_act(z, case["act"])[0]
        return {"y": y + d["res"] if "res" in d else y}
    if op == "lin_dx":
        dx, r = d["dy"] @ (d["w"] if flip else d["w"].t()), {}
        if case["z"] != "none":
            a, da = _x_act(_x_decode(s["z"]) if case["z"] == "act8" else d["z"], case["act"])
            dx = dx * da
            r = {"act_out": a} if case["act_out"] else {}
        return {"dx": dx + d["add"] if "add" in d else dx, **r}
    if op == "lin_dw":
        x = _x_decode(s["x"]) if case["x"] == "act8" else d["x"]
        dw = x.t() @ d["dy"]
        return {"dw": dw.t().contiguous() if flip else dw, **({"db": d["dy"].sum(0)} if case["db"] else {})}
    w1, w2 = (d["w1"].t(), d["w2"].t()) if flip else (d["w1"], d["w2"])
    xn, mean, rstd = _x_norm(d["x"], d["gain"], d["beta"])
    z = _x_round(xn, dt) @ w1 + d["b1"]
    h = _x_round(_x_act(z, case["act"])[0], dt)
    a, da = _x_act(_x_quant(z), case["act"])
    dz = _x_round((d["dy"] @ w2.t()) * da, dt)
    dw2, dw1 = _x_round(a, dt).t() @ d["dy"], _x_quant(xn).t() @ dz
    dx, dg, db = _x_norm_grad(_x_round(dz @ w1.t(), dt), d["x"], d["gain"], mean, rstd, d["dy"])
    return {"y": h @ w2 + d["b2"] + d["x"], "dx": dx, "dw1": dw1.t().contiguous() if flip else dw1,
            "dw2": dw2.t().contiguous() if flip else dw2, "db1": dz.sum(0), "db2": d["dy"].sum(0),
            "dgain": dg, "dbeta": db}
