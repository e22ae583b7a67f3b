"""Cases of the operators of a gated feed-forward block in training: the gated
projections with their three gradients, the norms before and after a block fused
with its gate, residual scales and dropout, and dropout by itself.  Each in a
plain form (elementary torch operations in float32) and as a caller of the
library runs it.

`own` selects: False computes the plain forms, True calls the library.
"""

import math

import torch

own = False

GROUP = 32          # columns that share one exponent of an 8-bit checkpoint
EPS = 1e-5
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
        # one token through the large layer: both weights are read once
        {"name": "gated fwd 1 4096-14336", "op": "g_fwd", "rows": 1, "in": 4096, "hid": 14336, "dtype": "bf16",
         "act": "silu", "bias": False, "keep": False, "layout": "out_in"},
        # the large layer's projections in training, both pre-activations kept for the backward pass
        {"name": "gated fwd 4096 4096-14336", "op": "g_fwd", "rows": 4096, "in": 4096, "hid": 14336, "dtype": "bf16",
         "act": "silu", "bias": False, "keep": True, "layout": "in_out"},
        # a small float32 model, GELU and biases
        {"name": "gated fwd 300 768-2048 f32", "op": "g_fwd", "rows": 300, "in": 768, "hid": 2048, "dtype": "f32",
         "act": "gelu", "bias": True, "keep": True, "layout": "in_out"},
        # gradient at both pre-activations through the down projection, from 8-bit checkpoints (ragged batch)
        {"name": "gated dh 4001 2816-1024 z8", "op": "g_dh", "rows": 4001, "hid": 2816, "out": 1024, "dtype": "bf16",
         "act": "silu", "z": "act8", "h": True, "layout": "in_out"},
        # input gradient: the sum of two products
        {"name": "gated dx 8192 1024-2816", "op": "g_dx", "rows": 8192, "in": 1024, "hid": 2816, "dtype": "bf16",
         "add": False, "layout": "in_out"},
        # both weight gradients of an expert-sized layer from the 8-bit layer input
        {"name": "gated dw 8192 2048-1408 x8", "op": "g_dw", "rows": 8192, "in": 2048, "hid": 1408, "dtype": "bf16",
         "x": "act8", "db": False, "dw": "bf16", "layout": "in_out"},
        # one decoding-sized batch between two blocks: launch latency
        {"name": "block norm fwd 16x768", "op": "n_fwd", "rows": 16, "cols": 768, "stream": "bf16", "dtype": "bf16",
         "params": "bf16", "branch": True, "post": "none", "pre": "rms", "gate": False, "alpha": 1.0, "beta": 1.0, "p": 0.0},
        # a float32 residual stream with an odd number of tokens; norms on both sides, gate and dropout
        {"name": "block norm fwd 8191x2048 f32 stream", "op": "n_fwd", "rows": 8191, "cols": 2048, "stream": "f32",
         "dtype": "bf16", "params": "f32", "branch": True, "post": "rms", "pre": "rms", "gate": True, "alpha": 1.0,
         "beta": 0.5, "p": 0.1},
        # the same between two blocks of a large layer, backward, with layer norms
        {"name": "block norm bwd 8192x4096", "op": "n_bwd", "rows": 8192, "cols": 4096, "stream": "bf16", "dtype": "bf16",
         "params": "bf16", "branch": True, "post": "layer", "pre": "layer", "gate": True, "alpha": 0.9, "beta": 0.5,
         "p": 0.1, "ds": True},
        # dropout of a large activation
        {"name": "dropout 16384x4096 bf16", "op": "drop", "rows": 16384, "cols": 4096, "dtype": "bf16", "p": 0.1,
         "add": False},
        # a small float32 one with the residual added
        {"name": "dropout 777x1001 f32 add", "op": "drop", "rows": 777, "cols": 1001, "dtype": "f32", "p": 0.25,
         "add": True},
        # a whole feed-forward block, forward and backward, with 8-bit checkpoints
        {"name": "ffn step 4096 1024-2816", "op": "ffn", "rows": 4096, "cols": 1024, "hid": 2816, "dtype": "bf16",
         "act": "silu", "post": "rms", "pre": "rms", "gate": True, "p": 0.1, "layout": "in_out"},
    ]


def _logint(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["g_fwd", "g_fwd", "g_dh", "g_dx", "g_dw", "n_fwd", "n_bwd", "drop", "ffn"])
    lay = rng.choice(["in_out", "out_in"])
    act = rng.choice(["silu", "silu", "gelu", "relu", "sigmoid"])
    if op in ("n_fwd", "n_bwd", "drop"):
        cols = _logint(rng, 64, 8192, 1 if rng.random() < 0.2 else 8)
        rows = _logint(rng, 1, min(16384, (1 << 26) // cols))
        stream, dt = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        c = {"op": op, "rows": rows, "cols": cols, "dtype": dt, "p": rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.9), 3)])}
        if op == "drop":
            c.update(add=rng.random() < 0.5)
            return c
        pre = rng.choice(["rms", "rms", "layer"])
        branch = rng.random() < 0.8
        post = rng.choice(["none", "rms", "rms", "layer"]) if branch else "none"
        c.update(stream=stream, params=rng.choice([dt, "f32"]), branch=branch, post=post, pre=pre,
                 gate=branch and rng.random() < 0.5, alpha=rng.choice([1.0, 0.75]) if branch else 1.0,
                 beta=rng.choice([1.0, 0.5]) if branch else 1.0)
        if not branch:
            c["p"] = 0.0
        if op == "n_bwd":
            c["ds"] = rng.random() < 0.8
        return c
    dt = "bf16" if op == "ffn" or rng.random() < 0.75 else "f32"
    budget = 4.0e11 if dt == "bf16" else 2.0e10
    step = 1 if rng.random() < 0.1 else 8
    nin, hid = _logint(rng, 128, 6144, step), _logint(rng, 128, 8192, step)
    if op == "ffn":
        cols, hid = _logint(rng, 128, 2048, 8), _logint(rng, 256, 6144, 8)
        rows = _logint(rng, 16, max(16, min(8192, int(budget / (18.0 * cols * hid)))))
        return {"op": op, "rows": rows, "cols": cols, "hid": hid, "dtype": dt, "act": act, "post": rng.choice(["none", "rms"]),
                "pre": rng.choice(["rms", "layer"]), "gate": rng.random() < 0.5, "p": rng.choice([0.0, 0.1]), "layout": lay}
    per = 2.0 * nin * hid * (1 if op == "g_dh" else 2)
    rows = _logint(rng, 1 if op == "g_fwd" else 16, max(16, min(16384, int(budget / per))))
    c = {"op": op, "rows": rows, "hid": hid, "dtype": dt, "layout": lay}
    if op == "g_fwd":
        c.update({"in": nin}, act=act, bias=rng.random() < 0.4, keep=rng.random() < 0.6)
    elif op == "g_dh":
        c.update(out=nin, act=act, z=rng.choice(["act8", "full"]), h=rng.random() < 0.7)
    elif op == "g_dx":
        c.update({"in": nin}, add=rng.random() < 0.4)
    else:
        c.update({"in": nin}, x=rng.choice(["act8", "full"]), db=rng.random() < 0.5, dw=rng.choice([dt, "f32"]))
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


def _stats(x, kind):
    """mean and 1 / root of a norm's rows (RMS: mean 0)."""
    xf = x.float()
    mean = xf.mean(1) if kind == "layer" else torch.zeros_like(xf[:, 0])
    return mean, (xf - mean[:, None]).square().mean(1).add(EPS).rsqrt()


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

    def weight(i, o, std, dtype=dt):
        return rnd(o, i, std=std, dtype=dtype) if case["layout"] == "out_in" else rnd(i, o, std=std, dtype=dtype)

    op, rows = case["op"], case["rows"]
    # a program's random state: a seed for the run, an offset for the layer and step
    s = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % 2 ** 64, "offset": seed % 1000003}
    f32 = torch.float32
    if op == "drop":
        n = case["cols"]
        s["x"], s["y"] = rnd(rows, n), out(rows, n)
        s["add"] = rnd(rows, n) if case["add"] else None
        return s
    if op in ("n_fwd", "n_bwd"):
        n, pt, st = case["cols"], _DT[case["params"]], _DT[case["stream"]]
        # a residual stream: rows of different sizes, a common offset
        s["x"] = (rnd(rows, n, dtype=f32) * rnd(rows, 1, dtype=f32).exp() + 0.3).to(st)
        for k in ("post", "pre"):
            s[k + "_gain"] = rnd(n, std=0.1, mean=1.0, dtype=pt) if case[k] != "none" else None
            s[k + "_bias"] = rnd(n, std=0.1, dtype=pt) if case[k] == "layer" else None
        s["gate"] = rnd(n, std=0.2, mean=0.5, dtype=pt) if case["gate"] else None
        s["branch"] = (rnd(rows, n, dtype=f32) * rnd(rows, 1, std=0.5, dtype=f32).exp()).to(dt) if case["branch"] else None
        if op == "n_fwd":
            s["s"], s["y"] = out(rows, n, dtype=st) if case["branch"] else None, out(rows, n)
            for k in ("post", "pre"):
                s[k + "_mean"] = out(rows, dtype=f32) if case[k] == "layer" else None
                s[k + "_rstd"] = out(rows, dtype=f32) if case[k] != "none" else None
            return s
        # x stands for the stream behind the junction here
        s["pre_mean"], s["pre_rstd"] = _stats(s["x"], case["pre"])
        if case["post"] != "none":
            s["post_mean"], s["post_rstd"] = _stats(s["branch"], case["post"])
        s["dy"] = rnd(rows, n, std=1e-2)
        s["ds"] = rnd(rows, n, std=1e-2, dtype=st) if case["ds"] else None
        s["dx"], s["dbranch"] = out(rows, n, dtype=st), out(rows, n) if case["branch"] else None
        for k in ("post_gain", "post_bias", "gate", "pre_gain", "pre_bias"):
            s["d" + k] = out(n, dtype=pt) if s[k] is not None else None
        return s
    if op == "ffn":
        n, f = case["cols"], case["hid"]
        s["x"], s["ds"], s["dy"] = rnd(rows, n), rnd(rows, n, std=1e-2), rnd(rows, n, std=1e-2)
        for k, on in (("g1", True), ("post_gain", case["post"] != "none"), ("g2", True)):
            s[k] = rnd(n, std=0.1, mean=1.0) if on else None
        for k in ("b1", "b2"):
            s[k] = rnd(n, std=0.1) if case["pre"] == "layer" else None
        s["gate"] = rnd(n, std=0.2, mean=0.5) if case["gate"] else None
        s["wg"], s["wu"], s["wd"] = weight(n, f, n ** -0.5), weight(n, f, n ** -0.5), weight(f, n, f ** -0.5)
        for k in ("wg", "wu", "wd", "g1", "b1", "g2", "b2", "post_gain", "gate"):
            s["d" + k] = torch.empty_like(s[k]) if s[k] is not None else None
        for k, c in (("n1", n), ("h", f), ("o", n), ("s", n), ("y", n), ("do", n), ("h2", f), ("dzg", f), ("dzu", f),
                     ("dn1", n), ("dxr", n), ("dx", n)):
            s[k] = out(rows, c)
        for k in ("m1", "r1", "rp", "m2", "r2"):
            s[k] = out(rows, dtype=f32)
        for k, c in (("n8", n), ("zg8", f), ("zu8", f)):
            s[k] = (out(rows, c, dtype=torch.int8), out(rows, -(-c // GROUP), dtype=torch.uint8))
        return s
    f = case["hid"]
    if op == "g_dh":
        o = case["out"]
        s["dy"], s["wd"] = rnd(rows, o, std=1e-2), weight(f, o, f ** -0.5)
        s["zg"], s["zu"] = rnd(rows, f, std=1.5), rnd(rows, f)
        if case["z"] == "act8":
            s["zg"], s["zu"] = _pack8(s["zg"]), _pack8(s["zu"])
        s["dzg"], s["dzu"], s["h"] = out(rows, f), out(rows, f), out(rows, f) if case["h"] else None
        return s
    k = case["in"]
    if op == "g_fwd":
        s["x"], s["wg"], s["wu"] = rnd(rows, k), weight(k, f, k ** -0.5), weight(k, f, k ** -0.5)
        s["bg"], s["bu"] = (rnd(f, std=0.1), rnd(f, std=0.1)) if case["bias"] else (None, None)
        s["h"] = out(rows, f)
        s["zg"], s["zu"] = (out(rows, f), out(rows, f)) if case["keep"] else (None, None)
        return s
    s["dzg"], s["dzu"] = rnd(rows, f, std=1e-2), rnd(rows, f, std=1e-2)
    if op == "g_dx":
        s["wg"], s["wu"] = weight(k, f, k ** -0.5), weight(k, f, k ** -0.5)
        s["add"], s["dx"] = rnd(rows, k, std=1e-2) if case["add"] else None, out(rows, k)
        return s
    s["x"] = rnd(rows, k)
    if case["x"] == "act8":
        s["x"] = _pack8(s["x"])
    shape = (f, k) if case["layout"] == "out_in" else (k, f)
    s["dwg"], s["dwu"] = out(*shape, dtype=_DT[case["dw"]]), out(*shape, dtype=_DT[case["dw"]])
    s["dbg"], s["dbu"] = (out(f), out(f)) if case["db"] else (None, None)
    return s


# ---- plain forms -------------------------------------------------------------

_MASK32 = 0xFFFFFFFF


def _kept(rows, cols, p, seed, offset, dev):
    """The dropout mask (kept elements) and the factor of what is kept.  Element
    (r, c) has 16 random bits, half c % 2 of word (c / 2) % 4 of the ten-round
    Philox 4x32 block (Salmon et al. 2011) of counter (c / 8, r, offset) under the
    key `seed`; it is dropped where they are under round(65536 p)."""
    t = int(round(p * 65536.0))
    c = [torch.arange(-(-cols // 8), dtype=torch.int64, device=dev)[None, :],
         torch.arange(rows, dtype=torch.int64, device=dev)[:, None],
         torch.full((1, 1), offset & _MASK32, dtype=torch.int64, device=dev),
         torch.full((1, 1), offset >> 32, dtype=torch.int64, device=dev)]
    k0, k1 = seed & _MASK32, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & _MASK32) ^ c[1] ^ k0, b & _MASK32, ((a >> 32) & _MASK32) ^ c[3] ^ k1, a & _MASK32]
        k0, k1 = (k0 + 0x9E3779B9) & _MASK32, (k1 + 0xBB67AE85) & _MASK32
    u = torch.stack([v for w in torch.broadcast_tensors(*c) for v in (w & 0xFFFF, w >> 16)], dim=2)
    scale = 65536.0 / (65536.0 - t) if t < 65536 else 0.0
    return (u.flatten(1)[:, :cols] >= t), scale


def _dropped(v, s, p):
    if p == 0.0:
        return v
    keep, scale = _kept(v.shape[0], v.shape[1], p, s["seed"], s["offset"], v.device)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _gate_act(z, kind):
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(_GELU_C * (z + 0.044715 * z * z * z)))
    if kind == "relu":
        return z.clamp_min(0.0)
    return torch.sigmoid(z)


def _gate_grad(z, kind):
    if kind == "silu":
        g = torch.sigmoid(z)
        return g * (1.0 + z * (1.0 - g))
    if kind == "gelu":
        t = torch.tanh(_GELU_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _GELU_C * (1.0 + 3 * 0.044715 * z * z)
    if kind == "relu":
        return (z > 0).float()
    g = torch.sigmoid(z)
    return g * (1.0 - g)


def _w_in_out(w, layout):
    return w.float().t() if layout == "out_in" else w.float()


def _norm(x, kind, gain, bias):
    """y (float32), mean, 1 / root"""
    mean, rstd = _stats(x, kind)
    y = (x.float() - mean[:, None]) * rstd[:, None]
    if gain is not None:
        y = y * gain.float()
    return (y if bias is None else y + bias.float()), mean, rstd


def _norm_grad(a, xh, rstd, kind):
    """gradient at a norm's input from a, the gradient at xh"""
    b = a - xh * (a * xh).mean(1, keepdim=True)
    if kind == "layer":
        b = b - a.mean(1, keepdim=True)
    return b * rstd[:, None]


def _junction(s, x, branch, st, dt, kind_post, kind_pre, alpha, beta, p, post_gain, post_bias, gate, pre_gain, pre_bias):
    """stream, y and the statistics of both norms"""
    pm = pr = None
    sn = x
    if branch is not None:
        t = branch.float()
        if kind_post != "none":
            t, pm, pr = _norm(branch, kind_post, post_gain, post_bias)
        t = _dropped(t, s, p)
        if gate is not None:
            t = t * gate.float()
        sn = (alpha * x.float() + beta * t).to(st)
    y, m, r = _norm(sn, kind_pre, pre_gain, pre_bias)
    return sn, y, pm, pr, m, r


def _junction_grad(s, case, dy, ds, sn, branch, st, dt, p, alpha, beta, q):
    """every gradient of a junction, each rounded once; q: parameters and statistics"""
    pt = q["pre_gain"].dtype
    dyf = dy.float()
    xh = (sn.float() - q["pre_mean"][:, None]) * q["pre_rstd"][:, None]
    g = _norm_grad(dyf * q["pre_gain"].float(), xh, q["pre_rstd"], case["pre"])
    if ds is not None:
        g = g + ds.float()
    r = {"dx": (alpha * g).to(st), "dpre_gain": (dyf * xh).sum(0).to(pt)}
    if q["pre_bias"] is not None:
        r["dpre_bias"] = dyf.sum(0).to(pt)
    if branch is None:
        return r
    e = beta * _dropped(g, s, p)
    gate = q["gate"].float() if q["gate"] is not None else 1.0
    if case["post"] == "none":
        t = branch.float()
        r["dbranch"] = (e * gate).to(dt)
    else:
        oh = (branch.float() - q["post_mean"][:, None]) * q["post_rstd"][:, None]
        gain = q["post_gain"].float()
        r["dbranch"] = _norm_grad(e * gate * gain, oh, q["post_rstd"], case["post"]).to(dt)
        r["dpost_gain"] = (e * gate * oh).sum(0).to(pt)
        t = oh * gain
        if q["post_bias"] is not None:
            r["dpost_bias"] = (e * gate).sum(0).to(pt)
            t = t + q["post_bias"].float()
    if q["gate"] is not None:
        r["dgate"] = (e * t).sum(0).to(pt)
    return r


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "drop":
        y = _dropped(s["x"].float(), s, case["p"])
        return {"y": (y if s["add"] is None else y + s["add"].float()).to(dt)}
    if op == "n_fwd":
        sn, y, pm, pr, m, r = _junction(s, s["x"], s["branch"], _DT[case["stream"]], dt, case["post"], case["pre"],
                                        case["alpha"], case["beta"], case["p"], s["post_gain"], s["post_bias"], s["gate"],
                                        s["pre_gain"], s["pre_bias"])
        o = {"y": y.to(dt), "pre_rstd": r}
        if case["branch"]:
            o["s"] = sn
        if case["pre"] == "layer":
            o["pre_mean"] = m
        if case["post"] != "none":
            o["post_rstd"] = pr
        if case["post"] == "layer":
            o["post_mean"] = pm
        return o
    if op == "n_bwd":
        return _junction_grad(s, case, s["dy"], s["ds"], s["x"], s["branch"], _DT[case["stream"]], dt, case["p"],
                              case["alpha"], case["beta"], s)
    lay = case["layout"]
    if op == "g_fwd":
        x = s["x"].float()
        zg, zu = x @ _w_in_out(s["wg"], lay), x @ _w_in_out(s["wu"], lay)
        if s["bg"] is not None:
            zg, zu = zg + s["bg"].float(), zu + s["bu"].float()
        r = {"h": (_gate_act(zg, case["act"]) * zu).to(dt)}
        return {**r, "zg": zg.to(dt), "zu": zu.to(dt)} if case["keep"] else r
    if op == "g_dh":
        dh = s["dy"].float() @ _w_in_out(s["wd"], lay).t()
        zg, zu = (_unpack8(*s["zg"]), _unpack8(*s["zu"])) if case["z"] == "act8" else (s["zg"].float(), s["zu"].float())
        a = _gate_act(zg, case["act"])
        r = {"dzg": (dh * zu * _gate_grad(zg, case["act"])).to(dt), "dzu": (dh * a).to(dt)}
        return {**r, "h": (a * zu).to(dt)} if case["h"] else r
    if op == "g_dx":
        dx = s["dzg"].float() @ _w_in_out(s["wg"], lay).t() + s["dzu"].float() @ _w_in_out(s["wu"], lay).t()
        return {"dx": (dx if s["add"] is None else dx + s["add"].float()).to(dt)}
    if op == "g_dw":
        x = _unpack8(*s["x"]) if case["x"] == "act8" else s["x"].float()
        r = {}
        for k in ("g", "u"):
            dz = s["dz" + k].float()
            r["dw" + k] = (dz.t() @ x if lay == "out_in" else x.t() @ dz).to(_DT[case["dw"]])
            if case["db"]:
                r["db" + k] = dz.sum(0).to(dt)
        return r
    # ffn: every operator rounds its result once; the backward pass sees the 8-bit checkpoints
    act, p = case["act"], case["p"]
    wg, wu, wd = (_w_in_out(s[k], lay) for k in ("wg", "wu", "wd"))
    _, n1, _, _, m1, r1 = _junction(s, s["x"], None, dt, dt, "none", case["pre"], 1.0, 1.0, 0.0, None, None, None, s["g1"],
                                    s["b1"])
    n8, n1 = _unpack8(*_pack8(n1)), n1.to(dt).float()
    zg, zu = n1 @ wg, n1 @ wu
    h = (_gate_act(zg, act) * zu).to(dt).float()
    zg8, zu8 = _unpack8(*_pack8(zg)), _unpack8(*_pack8(zu))
    o = (h @ wd).to(dt)
    sn, y, pm, pr, m2, r2 = _junction(s, s["x"], o, dt, dt, case["post"], case["pre"], 1.0, 0.5, p, s["post_gain"], None,
                                      s["gate"], s["g2"], s["b2"])
    q = {"pre_gain": s["g2"], "pre_bias": s["b2"], "pre_mean": m2, "pre_rstd": r2, "gate": s["gate"], "post_bias": None,
         "post_gain": s["post_gain"], "post_mean": pm, "post_rstd": pr}
    j = _junction_grad(s, case, s["dy"], s["ds"], sn, o, dt, dt, p, 1.0, 0.5, q)
    do = j["dbranch"].float()
    dh = do @ wd.t()
    a = _gate_act(zg8, act)
    dzg, dzu = (dh * zu8 * _gate_grad(zg8, act)).to(dt).float(), (dh * a).to(dt).float()
    h2 = (a * zu8).to(dt).float()
    dn1 = (dzg @ wg.t() + dzu @ wu.t()).to(dt)
    dwg, dwu, dwd = n8.t() @ dzg, n8.t() @ dzu, h2.t() @ do
    if lay == "out_in":
        dwg, dwu, dwd = (w.t().contiguous() for w in (dwg, dwu, dwd))
    q = {"pre_gain": s["g1"], "pre_bias": s["b1"], "pre_mean": m1, "pre_rstd": r1, "gate": None}
    k = _junction_grad(s, {"pre": case["pre"], "post": "none"}, dn1, j["dx"], s["x"], None, dt, dt, 0.0, 1.0, 1.0, q)
    r = {"s": sn, "y": y.to(dt), "dx": k["dx"], "dwg": dwg.to(dt), "dwu": dwu.to(dt), "dwd": dwd.to(dt),
         "dg1": k["dpre_gain"], "dg2": j["dpre_gain"]}
    if case["pre"] == "layer":
        r.update(db1=k["dpre_bias"], db2=j["dpre_bias"])
    if case["post"] != "none":
        r["dpost_gain"] = j["dpost_gain"]
    if case["gate"]:
        r["dgate"] = j["dgate"]
    return r


# ---- the library's calls -------------------------------------------------------

def _run_own(s):
    nsm, h = _lib()
    case = s["case"]
    op = case["op"]
    drop = nsm.Dropout(case["p"], s["seed"], s["offset"]) if case.get("p") else None
    if op == "drop":
        nsm.muon_dropout(h, s["x"], s["y"], drop or nsm.Dropout(0.0, 0), add=s["add"])
        return {"y": s["y"]}
    if op == "n_fwd":
        nsm.muon_blocknorm_forward(h, s["x"], branch=s["branch"], s=s["s"], y=s["y"], post_norm=case["post"],
                                   post_gain=s["post_gain"], post_bias=s["post_bias"], gate=s["gate"],
                                   pre_norm=case["pre"], pre_gain=s["pre_gain"], pre_bias=s["pre_bias"],
                                   residual_scale=case["alpha"], branch_scale=case["beta"], drop=drop, post_eps=EPS,
                                   pre_eps=EPS, post_mean=s["post_mean"], post_rstd=s["post_rstd"],
                                   pre_mean=s["pre_mean"], pre_rstd=s["pre_rstd"])
        return {k: s[k] for k in ("y", "pre_rstd", "s", "pre_mean", "post_rstd", "post_mean") if s[k] is not None}
    if op == "n_bwd":
        post = case["post"] != "none"
        nsm.muon_blocknorm_backward(h, s["dx"], ds=s["ds"], dy=s["dy"], s=s["x"], branch=s["branch"],
                                    dbranch=s["dbranch"], post_norm=case["post"], post_gain=s["post_gain"],
                                    post_bias=s["post_bias"], gate=s["gate"],
                                    post_mean=s["post_mean"] if case["post"] == "layer" else None,
                                    post_rstd=s["post_rstd"] if post else None, pre_norm=case["pre"],
                                    pre_gain=s["pre_gain"], pre_mean=s["pre_mean"] if case["pre"] == "layer" else None,
                                    pre_rstd=s["pre_rstd"], residual_scale=case["alpha"], branch_scale=case["beta"],
                                    drop=drop, dpost_gain=s["dpost_gain"], dpost_bias=s["dpost_bias"],
                                    dgate=s["dgate"], dpre_gain=s["dpre_gain"], dpre_bias=s["dpre_bias"])
        return {k: s[k] for k in ("dx", "dpre_gain", "dpre_bias", "dbranch", "dpost_gain", "dpost_bias", "dgate")
                if s[k] is not None}
    lay = case["layout"]
    if op == "g_fwd":
        nsm.muon_gated_forward(h, s["x"], s["wg"], s["wu"], s["h"], bias_gate=s["bg"], bias_up=s["bu"], act=case["act"],
                               gate_out=s["zg"], up_out=s["zu"], w_layout=lay)
        return {k: s[k] for k in ("h", "zg", "zu") if s[k] is not None}
    if op == "g_dh":
        zg, zu = (nsm.Act8(*s["zg"]), nsm.Act8(*s["zu"])) if case["z"] == "act8" else (s["zg"], s["zu"])
        nsm.muon_gated_grad_hidden(h, s["dy"], s["wd"], zg, zu, s["dzg"], s["dzu"], act=case["act"], h_out=s["h"],
                                   w_layout=lay)
        return {k: s[k] for k in ("dzg", "dzu", "h") if s[k] is not None}
    if op == "g_dx":
        nsm.muon_gated_grad_input(h, s["dzg"], s["dzu"], s["wg"], s["wu"], s["dx"], add=s["add"], w_layout=lay)
        return {"dx": s["dx"]}
    if op == "g_dw":
        x = nsm.Act8(*s["x"]) if case["x"] == "act8" else s["x"]
        nsm.muon_gated_grad_weight(h, x, s["dzg"], s["dzu"], s["dwg"], s["dwu"], db_gate=s["dbg"], db_up=s["dbu"],
                                   w_layout=lay)
        return {k: s[k] for k in ("dwg", "dbg", "dwu", "dbu") if s[k] is not None}
    act, pre, post = case["act"], case["pre"], case["post"]
    layer = pre == "layer"
    n8, zg8, zu8 = nsm.Act8(*s["n8"]), nsm.Act8(*s["zg8"]), nsm.Act8(*s["zu8"])
    m1, m2 = (s["m1"], s["m2"]) if layer else (None, None)
    rp = s["rp"] if post != "none" else None
    nsm.muon_blocknorm_forward(h, s["x"], y=s["n1"], pre_norm=pre, pre_gain=s["g1"], pre_bias=s["b1"], pre_eps=EPS,
                               pre_mean=m1, pre_rstd=s["r1"], y8=n8)
    nsm.muon_gated_forward(h, s["n1"], s["wg"], s["wu"], s["h"], act=act, gate_out=zg8, up_out=zu8, w_layout=lay)
    nsm.muon_linear_forward(h, s["h"], s["wd"], s["o"], w_layout=lay)
    nsm.muon_blocknorm_forward(h, s["x"], branch=s["o"], s=s["s"], y=s["y"], post_norm=post, post_gain=s["post_gain"],
                               gate=s["gate"], pre_norm=pre, pre_gain=s["g2"], pre_bias=s["b2"], branch_scale=0.5,
                               drop=drop, post_eps=EPS, pre_eps=EPS, post_rstd=rp, pre_mean=m2, pre_rstd=s["r2"])
    nsm.muon_blocknorm_backward(h, s["dxr"], ds=s["ds"], dy=s["dy"], s=s["s"], branch=s["o"], dbranch=s["do"],
                                post_norm=post, post_gain=s["post_gain"], gate=s["gate"], post_rstd=rp, pre_norm=pre,
                                pre_gain=s["g2"], pre_mean=m2, pre_rstd=s["r2"], branch_scale=0.5, drop=drop,
                                dpost_gain=s["dpost_gain"], dgate=s["dgate"], dpre_gain=s["dg2"], dpre_bias=s["db2"])
    nsm.muon_gated_grad_hidden(h, s["do"], s["wd"], zg8, zu8, s["dzg"], s["dzu"], act=act, h_out=s["h2"], w_layout=lay)
    nsm.muon_linear_grad_weight(h, s["h2"], s["do"], s["dwd"], w_layout=lay)
    nsm.muon_gated_grad_input(h, s["dzg"], s["dzu"], s["wg"], s["wu"], s["dn1"], w_layout=lay)
    nsm.muon_gated_grad_weight(h, n8, s["dzg"], s["dzu"], s["dwg"], s["dwu"], w_layout=lay)
    nsm.muon_blocknorm_backward(h, s["dx"], ds=s["dxr"], dy=s["dn1"], s=s["x"], pre_norm=pre, pre_gain=s["g1"],
                                pre_mean=m1, pre_rstd=s["r1"], dpre_gain=s["dg1"], dpre_bias=s["db1"])
    keys = ("s", "y", "dx", "dwg", "dwu", "dwd", "dg1", "dg2", "db1", "db2", "dpost_gain", "dgate")
    return {k: s[k] for k in keys if s[k] is not None}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    r, op = case["rows"], case["op"]
    if op == "drop":
        n = case["cols"]
        return {"bytes": (2 + case["add"]) * r * n * b, "flops": (2 + case["add"]) * r * n}
    if op in ("n_fwd", "n_bwd"):
        n = case["cols"]
        p, t = 2 if case["params"] == "bf16" else 4, 2 if case["stream"] == "bf16" else 4
        vec = sum((case["gate"], case["pre"] != "none", case["pre"] == "layer", case["post"] != "none",
                   case["post"] == "layer"))
        st = 4 * r * ((case["pre"] != "none") + (case["pre"] == "layer") + (case["post"] != "none") + (case["post"] == "layer"))
        if op == "n_fwd":
            return {"bytes": r * n * (t * (1 + case["branch"]) + b * (1 + case["branch"])) + vec * n * p + st,
                    "flops": r * n * (8 + 8 * case["branch"])}
        return {"bytes": r * n * (t * (2 + case["ds"]) + b * (1 + 2 * case["branch"])) + 2 * vec * n * p + st,
                "flops": r * n * (14 + 16 * case["branch"])}
    f = case["hid"]
    if op == "ffn":
        n = case["cols"]
        e8 = r * (n + -(-n // GROUP)) + 2 * r * (f + -(-f // GROUP))
        return {"bytes": b * (6 * r * n + 6 * n * f) + 2 * e8, "flops": 18 * r * n * f}
    if op == "g_dh":
        o = case["out"]
        z = 2 * b * r * f if case["z"] == "full" else 2 * r * (f + -(-f // GROUP))
        return {"bytes": b * (r * o + f * o + r * f * (2 + case["h"])) + z, "flops": 2 * r * f * o}
    k = case["in"]
    flops = 4 * r * k * f
    if op == "g_fwd":
        return {"bytes": b * (r * k + 2 * k * f + r * f * (3 if case["keep"] else 1) + 2 * f * case["bias"]), "flops": flops}
    if op == "g_dx":
        return {"bytes": b * (2 * r * f + 2 * k * f + r * k * (1 + case["add"])), "flops": flops}
    xb = b * r * k if case["x"] == "full" else r * (k + -(-k // GROUP))
    return {"bytes": xb + 2 * b * r * f + 2 * (2 if case["dw"] == "bf16" else 4) * k * f + 2 * b * f * case["db"],
            "flops": flops + 2 * r * f * case["db"]}


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


def _x_philox(words, key):
    """One block of ten rounds; 32-bit products from 16-bit halves."""
    def mul(a, m):
        lo, hi = a % 65536, a // 65536
        ml, mh = m % 65536, m // 65536
        mid = (lo * ml) // 65536 + (lo * mh) % 65536 + (hi * ml) % 65536
        low = (lo * ml) % 65536 + 65536 * (mid % 65536)
        return hi * mh + (lo * mh) // 65536 + (hi * ml) // 65536 + mid // 65536, low

    x0, x1, x2, x3 = words
    k0, k1 = key
    for i in range(10):
        h0, l0 = mul(x0, 0xD2511F53)
        h2, l2 = mul(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = (h2.bitwise_xor(x1).bitwise_xor((k0 + i * 0x9E3779B9) % 2 ** 32), l2,
                          h0.bitwise_xor(x3).bitwise_xor((k1 + i * 0xBB67AE85) % 2 ** 32), l0)
    return x0, x1, x2, x3


def _x_factor(rows, cols, p, s, dev):
    """0 for a dropped element, else what it is multiplied by."""
    cut = math.floor(p * 65536.0 + 0.5)
    if cut == 0:
        return torch.ones(rows, cols, dtype=torch.float64, device=dev)
    col = torch.arange(cols, device=dev)
    blocks = torch.arange((cols + 7) // 8, device=dev).expand(rows, -1)
    row = torch.arange(rows, device=dev)[:, None].expand_as(blocks)
    low, high = torch.full_like(row, s["offset"] % 2 ** 32), torch.full_like(row, s["offset"] // 2 ** 32)
    w = torch.stack(_x_philox((blocks, row, low, high), (s["seed"] % 2 ** 32, s["seed"] // 2 ** 32)))
    w = w[(col // 2) % 4, :, col // 8].t()
    bits = torch.where(col % 2 == 0, w % 65536, w // 65536)
    return (bits >= cut).double() * (65536.0 / max(65536 - cut, 1))


def _x_gate(z, kind):
    """(activation, derivative)"""
    if kind == "gelu":
        u = _GELU_C * (z + 0.044715 * z ** 3)
        sig = torch.sigmoid(2 * u)   # (1 + tanh u) / 2
        return z * sig, sig + z * 2 * sig * (1 - sig) * _GELU_C * (1 + 0.134145 * z ** 2)
    if kind == "relu":
        pos = (z > 0).double()
        return z * pos, pos
    sig = 1.0 / (1.0 + torch.exp(-z))
    return (z * sig, sig + z * sig * (1.0 - sig)) if kind == "silu" else (sig, sig * (1.0 - sig))


def _x_hat(x, kind):
    """(normalised rows, mean, 1 / root)"""
    n = x.shape[1]
    mean = x.sum(1, keepdim=True) / n if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1.0 / torch.sqrt((x - mean).pow(2).sum(1, keepdim=True) / n + EPS)
    return (x - mean) * rstd, mean[:, 0], rstd[:, 0]


def _x_affine(v, gain, bias):
    v = v if gain is None else v * gain
    return v if bias is None else v + bias


def _x_hat_grad(a, xh, rstd, kind):
    n = a.shape[1]
    proj = torch.einsum("ij,ij->i", a, xh)[:, None] / n
    shift = torch.einsum("ij->i", a)[:, None] / n if kind == "layer" else 0.0
    return (a - shift - proj * xh) * rstd[:, None]


def _x_junction(x, o, post, pre, alpha, beta, fac, d, st):
    """s, y and both norms' statistics; d: parameters"""
    pm = pr = None
    if o is not None:
        t = o
        if post != "none":
            t, pm, pr = _x_hat(o, post)
            t = _x_affine(t, d.get("post_gain"), d.get("post_bias"))
        t = t * fac * d["gate"] if "gate" in d else t * fac
        exact_s = alpha * x + beta * t
        x = _x_round(exact_s, st)
    else:
        exact_s = x
    yh, m, r = _x_hat(x, pre)
    return exact_s, x, _x_affine(yh, d.get("pre_gain"), d.get("pre_bias")), pm, pr, m, r


def _x_junction_grad(dy, ds, sv, o, post, pre, alpha, beta, fac, d):
    xh = (sv - d["pre_mean"][:, None]) * d["pre_rstd"][:, None]
    g = _x_hat_grad(d["pre_gain"] * dy, xh, d["pre_rstd"], pre)
    g = g if ds is None else g + ds
    r = {"dx": alpha * g, "dpre_gain": torch.einsum("ij,ij->j", dy, xh)}
    if "pre_bias" in d:
        r["dpre_bias"] = torch.einsum("ij->j", dy)
    if o is None:
        return r
    e = g * fac * beta
    eg = e * d["gate"] if "gate" in d else e
    if post == "none":
        t = o
        r["dbranch"] = eg
    else:
        oh = (o - d["post_mean"][:, None]) * d["post_rstd"][:, None]
        r["dbranch"] = _x_hat_grad(eg * d["post_gain"], oh, d["post_rstd"], post)
        r["dpost_gain"] = torch.einsum("ij,ij->j", eg, oh)
        if "post_bias" in d:
            r["dpost_bias"] = torch.einsum("ij->j", eg)
        t = _x_affine(oh, d["post_gain"], d.get("post_bias"))
    if "gate" in d:
        r["dgate"] = torch.einsum("ij,ij->j", e, t)
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = case["op"], _DT[case["dtype"]]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    rows = case["rows"]
    if op == "drop":
        y = d["x"] * _x_factor(rows, case["cols"], case["p"], s, d["x"].device)
        return {"y": y + d["add"] if "add" in d else y}
    if op in ("n_fwd", "n_bwd"):
        fac = _x_factor(rows, case["cols"], case["p"], s, d["x"].device) if case["branch"] else None
        args = (d.get("branch"), case["post"], case["pre"], case["alpha"], case["beta"], fac, d)
        if op == "n_bwd":
            return _x_junction_grad(d["dy"], d.get("ds"), d["x"], *args)
        sv, _, y, pm, pr, m, r = _x_junction(d["x"], *args, _DT[case["stream"]])
        o = {"y": y, "pre_rstd": r}
        if case["branch"]:
            o["s"] = sv
        if case["pre"] == "layer":
            o["pre_mean"] = m
        if case["post"] != "none":
            o["post_rstd"] = pr
        if case["post"] == "layer":
            o["post_mean"] = pm
        return o
    flip = case["layout"] == "out_in"

    def w(k):
        return d[k].t() if flip else d[k]

    if op == "g_fwd":
        zg, zu = d["x"] @ w("wg"), d["x"] @ w("wu")
        if "bg" in d:
            zg, zu = zg + d["bg"], zu + d["bu"]
        r = {"h": _x_gate(zg, case["act"])[0] * zu}
        return {**r, "zg": zg, "zu": zu} if case["keep"] else r
    if op == "g_dh":
        dh = d["dy"] @ w("wd").t()
        zg, zu = (_x_decode(s["zg"]), _x_decode(s["zu"])) if case["z"] == "act8" else (d["zg"], d["zu"])
        a, da = _x_gate(zg, case["act"])
        r = {"dzg": dh * da * zu, "dzu": a * dh}
        return {**r, "h": a * zu} if case["h"] else r
    if op == "g_dx":
        dx = torch.cat([d["dzg"], d["dzu"]], 1) @ torch.cat([w("wg"), w("wu")], 1).t()
        return {"dx": dx + d["add"] if "add" in d else dx}
    if op == "g_dw":
        x = _x_decode(s["x"]) if case["x"] == "act8" else d["x"]
        r = {}
        for k in ("g", "u"):
            dw = x.t() @ d["dz" + k]
            r["dw" + k] = dw.t().contiguous() if flip else dw
            if case["db"]:
                r["db" + k] = torch.einsum("ij->j", d["dz" + k])
        return r
    act, post, pre = case["act"], case["post"], case["pre"]
    p1 = {"pre_gain": d["g1"], **({"pre_bias": d["b1"]} if pre == "layer" else {})}
    p2 = {"pre_gain": d["g2"], **({"pre_bias": d["b2"]} if pre == "layer" else {}),
          **{k: d[k] for k in ("post_gain", "gate") if k in d}}
    _, _, n1, _, _, m1, r1 = _x_junction(d["x"], None, "none", pre, 1.0, 1.0, None, p1, dt)
    n8, nr = _x_quant(n1), _x_round(n1, dt)
    zg, zu = nr @ w("wg"), nr @ w("wu")
    h = _x_round(_x_gate(zg, act)[0] * zu, dt)
    o = _x_round(h @ w("wd"), dt)
    fac = _x_factor(rows, case["cols"], case["p"], s, o.device)
    sv, sr, y, pm, pr, m2, r2 = _x_junction(d["x"], o, post, pre, 1.0, 0.5, fac, p2, dt)
    p2.update(pre_mean=m2, pre_rstd=r2, post_mean=pm, post_rstd=pr)
    j = _x_junction_grad(d["dy"], d["ds"], sr, o, post, pre, 1.0, 0.5, fac, p2)
    do, dxr = _x_round(j["dbranch"], dt), _x_round(j["dx"], dt)
    a, da = _x_gate(_x_quant(zg), act)
    zu8 = _x_quant(zu)
    dh = do @ w("wd").t()
    dzg, dzu = _x_round(dh * da * zu8, dt), _x_round(dh * a, dt)
    dn1 = _x_round(dzg @ w("wg").t() + dzu @ w("wu").t(), dt)
    dws = {"dwg": n8.t() @ dzg, "dwu": n8.t() @ dzu, "dwd": _x_round(a * zu8, dt).t() @ do}
    p1.update(pre_mean=m1, pre_rstd=r1)
    k = _x_junction_grad(dn1, dxr, d["x"], None, "none", pre, 1.0, 1.0, None, p1)
    r = {"s": sv, "y": y, "dx": k["dx"], **{n: v.t().contiguous() if flip else v for n, v in dws.items()},
         "dg1": k["dpre_gain"], "dg2": j["dpre_gain"]}
    if pre == "layer":
        r.update(db1=k["dpre_bias"], db2=j["dpre_bias"])
    if post != "none":
        r["dpost_gain"] = j["dpost_gain"]
    if case["gate"]:
        r["dgate"] = j["dgate"]
    return r
