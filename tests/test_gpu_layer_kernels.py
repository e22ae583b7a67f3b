"""Every kernel the products' plan can pick, and the norm kernels over many rows
a workgroup, element by element against float64 on the GPU.

Bounds as in test_gpu_layers.py (u = 2^-24; h = half a step of a stored type): a
float32 sum of n products is off by at most (n + 16) u of the sum of their
magnitudes in any order, an activation adds 8 u (1 + |value|), its derivative
16 u of the product, and each output is rounded once.
"""

import pytest

import layer_plan_cases as cases

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_matrix_step_amd as m
    return m


@pytest.fixture(scope="module")
def h(nsm):
    hd = nsm.muon_init(0)
    yield hd
    nsm.muon_destroy(hd)


class Make:
    """Seeded device tensors of one type, all `shift` elements past a 16-byte boundary."""

    def __init__(self, seed, dt, shift):
        import torch
        self.torch, self.dt, self.shift = torch, dt, shift
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def blank(self, *shape, dt=None):
        n = 1
        for s in shape:
            n *= s
        return self.torch.full((n + self.shift,), 85.0, device="cuda", dtype=dt or self.dt)[self.shift:].view(*shape)

    def rnd(self, *shape, std=1.0, dt=None):
        t = self.blank(*shape, dt=dt)
        t.copy_(self.torch.empty(*shape, device="cuda").normal_(0, std, generator=self.g))
        return t

    def act8(self, nsm, r, c):
        q = self.torch.zeros(r * c + self.shift, device="cuda", dtype=self.torch.int8)[self.shift:].view(r, c)
        g = -(-c // 32)
        e = self.torch.zeros(r * g + self.shift, device="cuda", dtype=self.torch.uint8)[self.shift:].view(r, g)
        return nsm.Act8(q, e)

    def act8_of(self, nsm, x):
        """A checkpoint of x made here: the smallest exponent that keeps codes within 127."""
        torch, (r, c) = self.torch, x.shape
        a = self.act8(nsm, r, c)
        g = a.exponents.shape[1]
        p = torch.zeros(r, g * 32, device="cuda", dtype=torch.float64)
        p[:, :c] = x.double()
        p = p.view(r, g, 32)
        m, e = torch.frexp(p.abs().amax(dim=2) / 127.0)
        k = torch.where(m == 0.5, e - 1, e).clamp_min(-126)
        a.codes.copy_(torch.round(p * torch.exp2(-k.double())[..., None]).view(r, g * 32)[:, :c])
        a.exponents.copy_(k + 127)
        return a


def half(t):
    import torch
    return 2.0 ** -8 if t.dtype is torch.bfloat16 else 2.0 ** -24


def steps(a):
    import torch
    return torch.exp2(a.exponents.double() - 127).repeat_interleave(32, dim=1)[:, :a.codes.shape[1]]


def decoded(a):
    return a.codes.double() * steps(a)


def near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    if bool(bad.any()):
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {float(got[at])} for "
                             f"{float(want[at])}, bound {float(tol[at])}")


def near8(a, exact, tol, what):
    """A stored checkpoint of values known to `tol`: elements within half a step,
    and no group's step twice what its largest magnitude asks for."""
    import torch
    s = steps(a)
    near(decoded(a), exact, s / 2 + tol, what)
    r, c = exact.shape
    top = torch.zeros(r, a.exponents.shape[1] * 32, device="cuda", dtype=torch.float64)
    top[:, :c] = exact.abs() + tol
    top = top.view(r, -1, 32).amax(dim=2)
    e = a.exponents.double()
    assert bool(((e == 1) | (top >= 63.5 * torch.exp2(e - 127))).all()), f"{what}: exponents"


def act(z, kind):
    """(value, derivative) in float64"""
    import torch
    if kind == "gelu":
        k = (2.0 / torch.pi) ** 0.5
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if kind == "relu_sq":
        r = z.clamp_min(0.0)
        return r * r, 2 * r
    return z, torch.ones_like(z)


def parse(line):
    import torch
    w = line.split()
    r, a, b = (int(v) for v in w[1:4])
    dt = torch.float32 if "f32" in w else torch.bfloat16
    return w[0], r, a, b, dt, "out_in" if "oi" in w else "in_out", 1 if "shift=1" in w else 0, "x8" in w


def check_forward(nsm, h, line):
    _, rows, k, n, dt, layout, shift, _ = parse(line)
    m = Make(rows + k + n, dt, shift)
    x, w = m.rnd(rows, k), m.rnd(*((n, k) if layout == "out_in" else (k, n)), std=k ** -0.5)
    wio = (w.t() if layout == "out_in" else w).double().contiguous()
    prod, mag = x.double() @ wio, x.double().abs() @ wio.abs()
    bias, res = m.rnd(n), m.rnd(rows, n)
    d = (k + 16) * U * (mag + bias.double().abs())

    y, zt = m.blank(rows, n), m.blank(rows, n)
    nsm.muon_linear_forward(h, x, w, y, bias=bias, act="gelu", residual=res, z_out=zt, w_layout=layout)
    z = prod + bias.double()
    near(zt, z, d + half(zt) * z.abs(), "z")
    want = act(z, "gelu")[0] + res.double()
    near(y, want, 1.2 * d + 8 * U * (1 + want.abs()) + 2 * U * res.double().abs() + (4 * U + half(y)) * want.abs(), "y, gelu")

    y.copy_(res)
    z8 = m.act8(nsm, rows, n)
    nsm.muon_linear_forward(h, x, w, y, act="relu_sq", residual=y, z_out=z8, w_layout=layout)
    d = (k + 16) * U * mag
    near8(z8, prod, d, "z8")
    want = act(prod, "relu_sq")[0] + res.double()
    near(y, want, (2 * prod.abs() + d) * d + 2 * U * res.double().abs() + (6 * U + half(y)) * want.abs() +
         4 * U * (want - res.double()).abs(), "y, relu_sq, in place")

    nsm.muon_linear_forward(h, x, w, y, w_layout=layout)
    near(y, prod, d + half(y) * prod.abs(), "y, plain")


def check_grad_input(nsm, h, line):
    _, rows, k, n, dt, layout, shift, _ = parse(line)
    m = Make(rows + k + n, dt, shift)
    dy, w = m.rnd(rows, n), m.rnd(*((n, k) if layout == "out_in" else (k, n)), std=n ** -0.5)
    wt = (w if layout == "out_in" else w.t()).double().contiguous()
    prod, mag = dy.double() @ wt, dy.double().abs() @ wt.abs()
    z, add = m.rnd(rows, k, std=2.0), m.rnd(rows, k)
    d = (n + 16) * U * mag

    def check(dx, v, zv, kind, av, what):
        val, der = act(zv, kind)
        want = prod * der + av
        near(dx, want, d * der.abs() + 16 * U * prod.abs() * (1 + der.abs()) + 2 * U * (av.abs() + want.abs()) +
             half(dx) * want.abs(), f"dx, {what}")
        near(v, val, 8 * U * (1 + val.abs()) + half(v) * val.abs(), f"act_out, {what}")

    dx, v = m.blank(rows, k), m.blank(rows, k)
    nsm.muon_linear_grad_input(h, dy, w, dx, act="gelu", z=z, act_out=v, add=add, w_layout=layout)
    check(dx, v, z.double(), "gelu", add.double(), "gelu")
    z8 = m.act8_of(nsm, z)
    dx.copy_(add)
    v.fill_(85.0)
    nsm.muon_linear_grad_input(h, dy, w, dx, act="relu_sq", z=z8, act_out=v, add=dx, w_layout=layout)
    check(dx, v, decoded(z8), "relu_sq", add.double(), "relu_sq, 8 bits, in place")
    nsm.muon_linear_grad_input(h, dy, w, dx, w_layout=layout)
    near(dx, prod, d + half(dx) * prod.abs(), "dx, plain")


def check_grad_weight(nsm, h, line):
    import torch
    _, rows, k, n, dt, layout, shift, x8 = parse(line)
    m = Make(rows + k + n, dt, shift)
    xf, dy = m.rnd(rows, k), m.rnd(rows, n)
    x = m.act8_of(nsm, xf) if x8 else xf
    xv, dyv = decoded(x) if x8 else xf.double(), dy.double()
    want, mag = xv.t().contiguous() @ dyv, xv.abs().t().contiguous() @ dyv.abs()
    if layout == "out_in":
        want, mag = want.t(), mag.t()
    sums, smag = dyv.sum(0), dyv.abs().sum(0)
    other = torch.bfloat16 if dt is torch.float32 else torch.float32
    for acc, dwt, dbt in ((True, dt, torch.float32), (False, other, torch.bfloat16)):
        dw, db = m.rnd(*want.shape, dt=dwt), m.rnd(n, dt=dbt)
        w0, b0 = (dw.double(), db.double()) if acc else (torch.zeros_like(want), torch.zeros_like(sums))
        nsm.muon_linear_grad_weight(h, x, dy, dw, db=db, accumulate=acc, w_layout=layout)
        r = want + w0
        near(dw, r, (rows + 16) * U * mag + 2 * U * w0.abs() + (4 * U + half(dw)) * r.abs(), f"dw, accumulate {acc}")
        r = sums + b0
        near(db, r, (rows + 16) * U * smag + 2 * U * b0.abs() + (2 * U + half(db)) * r.abs(), f"db, accumulate {acc}")
    dw = m.blank(*want.shape)
    nsm.muon_linear_grad_weight(h, x, dy, dw, w_layout=layout)
    near(dw, want, (rows + 16) * U * mag + (4 * U + half(dw)) * want.abs(), "dw alone")


CHECKS = {"fwd": check_forward, "dx": check_grad_input, "dw": check_grad_weight}


@pytest.mark.parametrize("line", cases.CASES + cases.STREAMS)
def test_product_kernel(nsm, h, line):
    CHECKS[line.split()[0]](nsm, h, line)


# Rows of 2, 4 and 8 waves (and one of 32 elements a lane), in vectors and not,
# enough of them that each workgroup takes at least three rows forward and six
# backward, the last turn ragged: 512 workgroups of 4, 2 or 1 rows forward, 256
# backward.  Then outputs over and under the size from which they are streamed,
# for each number of waves and both types.
NORM_SHAPES = [(7001, 2048), (7001, 1030), (3501, 4096), (3501, 4095), (1801, 8192), (1801, 8191), (1801, 12288),
               (1801, 9001), (18001, 1000), (9001, 2048), (4500, 4096), (2200, 8192), (5000, 776), (3001, 2048),
               (1201, 4096), (700, 8192), (300, 12288)]


def depth(cols):
    """Additions one after the other in a row's sum (test_gpu_layers.py)."""
    return 64 + cols / 512


@pytest.mark.parametrize("st,pst", [("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm_over_many_rows(nsm, h, rows, cols, st, pst):
    import torch
    types = {"bf16": torch.bfloat16, "fp32": torch.float32}
    m, pt = Make(rows + cols, types[st], 0), types[pst]
    x = m.rnd(rows, cols)
    x *= m.rnd(rows, 1).exp()
    x += 0.5
    gain, bias = m.rnd(cols, dt=pt), m.rnd(cols, dt=pt)
    xv, gv, bv = x.double(), gain.double(), bias.double()
    y, y8 = m.blank(rows, cols), m.act8(nsm, rows, cols)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    eps = torch.tensor(1e-5, dtype=torch.float32).double().item()
    nsm.muon_layernorm_forward(h, x, gain, bias, y, mean=mean, rstd=rstd, eps=eps, y8=y8)
    mu = xv.mean(1)
    r = ((xv - mu[:, None]).square().mean(1) + eps).rsqrt()
    xh, mag, d = (xv - mu[:, None]) * r[:, None], xv.abs().mean(1), depth(cols) * U
    near(mean, mu, d * mag + U * mu.abs(), "mean")
    near(rstd, r, (d + (d * mag * r) ** 2) * r, "rstd")
    want = xh * gv + bv
    tol = 2 * d * (gv.abs() * (xh.abs() + (r * mag)[:, None]) + bv.abs()) + 4 * U * want.abs()
    near(y, want, tol + half(y) * want.abs(), "y")
    near8(y8, want, tol, "y8")

    mv, rv = mean.double(), rstd.double()
    xh = (xv - mv[:, None]) * rv[:, None]
    dy, add = m.rnd(rows, cols), m.rnd(rows, cols)
    a = dy.double() * gv
    base = rv[:, None] * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    dtol = 2 * d * rv[:, None] * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True))
    sums = ((dy.double() * xh).sum(0), dy.double().sum(0))
    smag = ((dy.double() * xh).abs().sum(0), dy.double().abs().sum(0))
    for in_place in (False, True):
        dx, dg, db = m.blank(rows, cols), m.rnd(cols, dt=pt), m.rnd(cols, dt=pt)
        if in_place:
            dx.copy_(add)
        g0 = [t.double() if in_place else torch.zeros_like(gv) for t in (dg, db)]
        nsm.muon_layernorm_backward(h, dy, x, gain, mean, rstd, dx, dg, dbias=db, add=dx if in_place else add,
                                    accumulate=in_place)
        want = base + add.double()
        near(dx, want, dtol + 4 * U * (want.abs() + add.double().abs()) + half(dx) * want.abs(), f"dx, in place {in_place}")
        for got, s, g, mg, what in ((dg, sums[0], g0[0], smag[0], "dgain"), (db, sums[1], g0[1], smag[1], "dbias")):
            near(got, s + g, (rows + 64) * U * mg + 2 * U * g.abs() + (U + half(got)) * (s + g).abs(), what)
