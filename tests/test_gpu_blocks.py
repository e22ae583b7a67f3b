"""GPU parity of the block operators through the C ABI against the float64 oracle,
element by element.

Bounds (u = 2^-24, the float32 unit roundoff; h = half a step of the result's type
relative to it, 2^-8 for bf16 and 2^-24 for float32):

  - a float32 sum of n products is off by at most (n + 8) u times the sum of their
    magnitudes, in any order; an element of such a sum that is itself off by e adds e;
  - a norm's row sums run through at most D = 64 + cols / 512 additions one after the
    other (a lane's elements, the lanes, the waves; a layer norm's waves centre their
    own columns, whose squares join through one product more each), so a mean is off by
    D u mean|.| and 1 / root by D u relative;
  - a gate adds at most 8 u (1 + |value|), its derivative 16 u (rounding of its
    argument times the logistic's slope, a few units of arithmetic), and no gate's
    slope passes 1.13;
  - each product or sum of two in an epilogue adds u relative; each output is rounded
    once: h |result|.
"""

import numpy as np
import pytest

from oracle import block_oracle as bo
from oracle import layer_oracle as lo
from test_gpu_layers import HALF, U, act8_blank, act8_dev, blank, check_act8, close, dev, host, padding_kept

pytestmark = pytest.mark.gpu
SLOPE = 1.13


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_matrix_step_amd as m
    return m


@pytest.fixture()
def h(nsm):
    hd = nsm.muon_init(0)
    yield hd
    nsm.muon_destroy(hd)


def same_ld(a, b):
    return a.stride(0) == b.stride(0)


# ---- gated feed-forward -----------------------------------------------------------

def gated_case(rows, i, f, st, lay, pad, shift, seed=1):
    rng = np.random.default_rng([seed, rows, i, f])
    shape = (f, i) if lay == "out_in" else (i, f)
    x = dev(rng.normal(size=(rows, i)), st, pad, shift)
    wg, wu = (dev(rng.normal(size=shape) / np.sqrt(i), st, pad, shift) for _ in range(2))
    return rng, x, wg, wu


# rows, in, hidden, type, layout, padding, shift: every tile edge, ragged sizes, one token, misaligned rows
GATED = [(1, 256, 96, "bf16", "in_out", 0, 0), (1, 1024, 1408, "bf16", "out_in", 0, 0), (5, 72, 40, "bf16", "in_out", 8, 0),
         (33, 100, 77, "bf16", "out_in", 3, 1), (130, 200, 136, "bf16", "in_out", 0, 0), (300, 136, 264, "bf16", "out_in", 0, 8),
         (64, 1, 1, "bf16", "in_out", 0, 0), (1000, 520, 1000, "bf16", "in_out", 0, 0), (2050, 320, 1416, "bf16", "out_in", 0, 0),
         (3000, 136, 2000, "bf16", "in_out", 0, 0), (1, 64, 33, "fp32", "in_out", 0, 0), (70, 97, 130, "fp32", "out_in", 1, 1),
         (300, 256, 520, "fp32", "in_out", 0, 0), (1030, 64, 700, "fp32", "out_in", 4, 0)]


@pytest.mark.parametrize("act,keep,bias", [("silu", "full", True), ("gelu", "8", False), ("sigmoid", "none", True),
                                           ("relu", "8", True)])
@pytest.mark.parametrize("case", GATED, ids=str)
def test_gated_forward(nsm, h, case, act, keep, bias):
    rows, i, f, st, lay, pad, shift = case
    rng, (x, xv), (wg, wgv), (wu, wuv) = gated_case(rows, i, f, st, lay, pad, shift)
    bg = dev(rng.normal(size=f), st, 0, shift) if bias else (None, None)
    bu = dev(rng.normal(size=f), st, 0, shift) if bias else (None, None)
    y = blank(rows, f, st, pad, shift)
    zo = {"none": (None, None), "full": (blank(rows, f, st, pad, shift), blank(rows, f, st, pad, shift)),
          "8": (act8_blank(nsm, rows, f, pad, shift), act8_blank(nsm, rows, f, pad, shift))}[keep]
    nsm.muon_gated_forward(h, x, wg, wu, y, bias_gate=bg[0], bias_up=bu[0], act=act, gate_out=zo[0], up_out=zo[1],
                           w_layout=lay)
    want, zg, zu = bo.gated(xv, wgv, wuv, bg[1], bu[1], act, lay)
    tz = [(i + 8) * U * (np.abs(xv) @ np.abs(lo.weight_in_out(w, lay))) + 2 * U * np.abs(z) +
          (0 if b is None else 2 * U * np.abs(b)) for w, z, b in ((wgv, zg, bg[1]), (wuv, zu, bu[1]))]
    a = np.abs(bo.gate(zg, act)[0])
    ta = SLOPE * tz[0] + 8 * U * (1 + a)
    close(host(y), want, ta * np.abs(zu) + (a + ta) * tz[1] + (2 * U + HALF[st]) * np.abs(want), "h")
    assert padding_kept(y)
    if keep == "full":
        for z, v, t, nm in ((zo[0], zg, tz[0], "gate"), (zo[1], zu, tz[1], "up")):
            close(host(z), v, t + HALF[st] * np.abs(v), nm)
            assert padding_kept(z)
    if keep == "8":
        check_act8(zo[0], zg, tz[0], "gate8")
        check_act8(zo[1], zu, tz[1], "up8")
        assert all(padding_kept(q.codes) and padding_kept(q.exponents) for q in zo)


@pytest.mark.parametrize("act,z8,with_h", [("silu", True, True), ("gelu", False, True), ("sigmoid", True, False),
                                           ("relu", False, True)])
@pytest.mark.parametrize("case", GATED, ids=str)
def test_gated_grad_hidden(nsm, h, case, act, z8, with_h):
    rows, o, f, st, lay, pad, shift = case
    rng = np.random.default_rng([2, rows, o, f])
    dy, dyv = dev(rng.normal(size=(rows, o)), st, pad, shift)
    wd, wdv = dev(rng.normal(size=(o, f) if lay == "out_in" else (f, o)) / np.sqrt(f), st, pad, shift)
    zv = [rng.normal(size=(rows, f)) * 1.5, rng.normal(size=(rows, f))]
    if z8:
        (zg, zgv), (zu, zuv) = (act8_dev(nsm, v, pad, shift) for v in zv)
    else:
        (zg, zgv), (zu, zuv) = (dev(v, st, pad, shift) for v in zv)
    dg, du, ho = (blank(rows, f, st, pad, shift) for _ in range(3))
    nsm.muon_gated_grad_hidden(h, dy, wd, zg, zu, dg, du, act=act, h_out=ho if with_h else None, w_layout=lay)
    wdg, wdu, wh, dh = bo.gated_grad_hidden(dyv, wdv, zgv, zuv, act, lay)
    a, d = (np.abs(v) for v in bo.gate(zgv, act))
    td = (o + 8) * U * (np.abs(dyv) @ np.abs(lo.weight_in_out(wdv, lay)).T)
    ta, h_ = 8 * U * (1 + a), HALF[st]
    close(host(dg), wdg, np.abs(zuv) * (td * (d + 16 * U) + np.abs(dh) * 16 * U) + (3 * U + h_) * np.abs(wdg), "dgate")
    close(host(du), wdu, td * (a + ta) + np.abs(dh) * ta + (2 * U + h_) * np.abs(wdu), "dup")
    assert padding_kept(dg) and padding_kept(du)
    if with_h:
        close(host(ho), wh, ta * np.abs(zuv) + (2 * U + h_) * np.abs(wh), "h")
        assert padding_kept(ho)


@pytest.mark.parametrize("add", [None, "other", "itself"])
@pytest.mark.parametrize("case", GATED, ids=str)
def test_gated_grad_input(nsm, h, case, add):
    rows, i, f, st, lay, pad, shift = case
    rng, (_, _), (wg, wgv), (wu, wuv) = gated_case(rows, i, f, st, lay, pad, shift)
    (dg, dgv), (du, duv) = (dev(rng.normal(size=(rows, f)), st, pad, shift) for _ in range(2))
    dx = blank(rows, i, st, pad, shift)
    av = None
    ad = None
    if add:
        ad, av = dev(rng.normal(size=(rows, i)), st, pad, shift)
        if add == "itself":
            dx = ad
    nsm.muon_gated_grad_input(h, dg, du, wg, wu, dx, add=ad, w_layout=lay)
    want = bo.gated_grad_input(dgv, duv, wgv, wuv, av, lay)
    mag = np.abs(dgv) @ np.abs(lo.weight_in_out(wgv, lay)).T + np.abs(duv) @ np.abs(lo.weight_in_out(wuv, lay)).T
    close(host(dx), want, (2 * f + 8) * U * mag + (2 * U + HALF[st]) * np.abs(want) + (0 if av is None else U * np.abs(av)), "dx")
    assert add == "itself" or padding_kept(dx)


@pytest.mark.parametrize("x8,db,acc,dwt", [(False, "both", False, "same"), (True, "up", True, "fp32"), (True, "none", False, "same"),
                                           (False, "gate", True, "same")])
@pytest.mark.parametrize("case", GATED, ids=str)
def test_gated_grad_weight(nsm, h, case, x8, db, acc, dwt):
    rows, i, f, st, lay, pad, shift = case
    wt = st if dwt == "same" else dwt
    rng = np.random.default_rng([3, rows, i, f])
    x, xv = act8_dev(nsm, rng.normal(size=(rows, i)), pad, shift) if x8 else dev(rng.normal(size=(rows, i)), st, pad, shift)
    (dg, dgv), (du, duv) = (dev(rng.normal(size=(rows, f)), st, pad, shift) for _ in range(2))
    shape = (f, i) if lay == "out_in" else (i, f)
    dw = [dev(rng.normal(size=shape), wt, pad, shift) for _ in range(2)]
    b = [dev(rng.normal(size=f), "fp32", 0, shift) if db in ("both", k) else (None, None) for k in ("gate", "up")]
    nsm.muon_gated_grad_weight(h, x, dg, du, dw[0][0], dw[1][0], db_gate=b[0][0], db_up=b[1][0], accumulate=acc, w_layout=lay)
    for (w, w0), (v, v0), dz, nm in ((dw[0], b[0], dgv, "gate"), (dw[1], b[1], duv, "up")):
        want, wb = lo.linear_grad_weight(xv, dz, lay)
        mag = np.abs(xv).T @ np.abs(dz)
        mag = mag.T if lay == "out_in" else mag
        old = w0 if acc else 0.0
        close(host(w), want + old, (rows + 8) * U * mag + (2 * U + HALF[wt]) * np.abs(want + old) + U * np.abs(old), "dw " + nm)
        if v is not None:
            old = v0 if acc else 0.0
            close(host(v), wb + old, (rows + 8) * U * np.abs(dz).sum(0) + 2 * U * (np.abs(wb + old) + np.abs(old)), "db " + nm)


def test_gates_at_infinities_and_nan(nsm, h):
    """An identity weight carries the pre-activations through: limits and NaN of every
    gate, forward and backward, in the epilogues of interior and of ragged tiles."""
    import torch
    vals = [0.0, -0.0, 1.0, -1.0, 9.5, -9.5, 79.0, -79.0, 81.0, -81.0, 200.0, -200.0, 3e4, -3e4, float("inf"), float("-inf"),
            float("nan")]
    for f in (64, 60):
        z = torch.tensor([vals[(r * 7 + c) % len(vals)] for r in range(64) for c in range(f)]).view(64, f).cuda()
        one = torch.ones(64, f, device="cuda")
        zv, dy = z.double().cpu().numpy(), torch.eye(64, device="cuda")
        wd = torch.ones(f, 64, device="cuda")        # dh = 1
        for act in nsm.GATES:
            out = [torch.empty(64, f, device="cuda") for _ in range(3)]
            nsm.muon_gated_grad_hidden(h, dy, wd, z, one, *out[:2], act=act, h_out=out[2])
            with np.errstate(all="ignore"):
                a, d = bo.gate(np.where(np.isinf(zv), 0, zv), act)
            lim = {"silu": (np.inf, 1, 0, 0), "gelu": (np.inf, 1, 0, 0), "relu": (np.inf, 1, 0, 0), "sigmoid": (1, 0, 0, 0)}[act]
            for s, (va, vd) in ((np.inf, lim[:2]), (-np.inf, lim[2:])):
                a, d = np.where(zv == s, va, a), np.where(zv == s, vd, d)
            for got, want in ((out[1], a), (out[2], a), (out[0], d)):
                g = host(got)
                assert (np.isnan(g) == np.isnan(zv)).all(), act
                fin = np.isfinite(want) & ~np.isnan(zv)
                assert (g[np.isinf(want)] == want[np.isinf(want)]).all(), act
                close(g[fin], want[fin], 16 * U * (1 + np.abs(want[fin])), act)


def test_gated_rows_far_apart(nsm, h):
    """Rows whose offsets pass 2^31 elements."""
    import torch
    rows, ld = 70000, 32768
    big = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    x = big[:, 64:128]
    x.normal_()
    hd = big[:, 4096:4128]
    w = torch.randn(64, 32, device="cuda").bfloat16()
    nsm.muon_gated_forward(h, x, w, w, hd, act="relu")     # one weight for both projections
    z = x.float() @ w.float()
    want = z.clamp_min(0) * z
    assert float(((hd.float() - want).abs() - 2.0 ** -8 * want.abs()).max()) < 1e-3


# ---- dropout ------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols,st,pad,shift", [(1, 1, "bf16", 0, 0), (3, 31, "fp32", 0, 0), (17, 1000, "bf16", 0, 0),
                                                    (40, 1001, "bf16", 0, 1), (40, 999, "fp32", 3, 1), (1200, 24, "bf16", 8, 0),
                                                    (5, 9000, "fp32", 0, 0), (2100, 3, "bf16", 0, 0)])
@pytest.mark.parametrize("p,add", [(0.1, None), (0.5, "other"), (0.0, "itself"), (1.0, "other"), (0.93, None)])
def test_dropout(nsm, h, rows, cols, st, pad, shift, p, add):
    rng = np.random.default_rng([4, rows, cols])
    x, xv = dev(rng.normal(size=(rows, cols)), st, pad, shift)
    y = blank(rows, cols, st, pad, shift)
    ad, av = dev(rng.normal(size=(rows, cols)), st, pad, shift) if add else (None, 0.0)
    if add == "itself":
        y = ad
    seed, offset = 0xFEDCBA9876543210, (3 << 40) + 17
    nsm.muon_dropout(h, x, y, nsm.Dropout(p, seed, offset), add=ad)
    f = bo.dropout_factors(rows, cols, p, seed, offset)
    want = xv * f
    close(host(y), want + av, 2 * U * np.abs(want) + U * np.abs(want + av) + HALF[st] * np.abs(want + av), "y")
    assert add == "itself" or padding_kept(y)
    nsm.muon_dropout(h, x, x, nsm.Dropout(p, seed, offset))      # in place
    close(host(x), want, (2 * U + HALF[st]) * np.abs(want), "in place")


def test_dropped_infinities_and_nan_become_zero(nsm, h):
    import torch
    x = torch.full((64, 256), float("nan"), device="cuda")
    x[:, ::2] = float("inf")
    y = torch.empty_like(x)
    nsm.muon_dropout(h, x, y, nsm.Dropout(0.5, 9))
    keep = torch.from_numpy(bo.dropout_factors(64, 256, 0.5, 9, 0) != 0).cuda()
    assert bool((y[~keep] == 0).all()) and bool(torch.isnan(y[keep & torch.isnan(x)]).all())
    assert bool((y[keep & torch.isinf(x)] == float("inf")).all())


def test_dropout_rows_far_apart(nsm, h):
    import torch
    rows, ld = 70000, 32768
    big = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    x, y = big[:, :40], big[:, 100:140]
    x.fill_(1.0)
    nsm.muon_dropout(h, x, y, nsm.Dropout(0.25, 77, 5))
    f = bo.dropout_factors(rows, 40, 0.25, 77, 5)
    assert ((host(y) != 0) == (f != 0)).all()


def test_captured_dropout_counts_steps(nsm, h):
    """Every replay draws the mask of the step that the program's counter holds."""
    import torch
    x = torch.ones(37, 130, device="cuda")
    y = torch.empty_like(x)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = nsm.Dropout(0.3, 21, 100, step=step)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nsm.muon_dropout(h, x, y, drop)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        nsm.muon_dropout(h, x, y, drop)
        step.add_(1)
    for n in range(4):
        y.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = bo.dropout_factors(37, 130, 0.3, 21, 100 + n)
        close(host(y), want, 2 * U * want, f"replay {n}")
    assert int(step) == 4


# ---- norms around a block --------------------------------------------------------------

def depth(cols):
    return 64 + cols / 512


TYPES = [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")]
# rows, cols: one to sixteen waves a row, ragged rows, rows longer than the registers
SHAPES = [(1, 1), (3, 40), (37, 513), (9, 1000), (600, 1024), (5, 1501), (6, 2048), (1100, 2047), (3, 4096), (5, 5000),
          (2, 8192), (530, 8191), (3, 9001), (1030, 8200)]


def junction(rng, rows, cols, sst, bst, pst, post, pre, gate, branch, pad, shift):
    t = {"x": dev(rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1))) + 0.3, sst, pad, shift)}
    if branch:
        t["branch"] = dev(rng.normal(size=(rows, cols)) + 0.2, bst, pad, shift)
    for k, on in (("post_gain", post != "none"), ("post_bias", post == "layer"), ("gate", gate), ("pre_gain", pre != "none"),
                  ("pre_bias", pre == "layer")):
        if on:
            t[k] = dev(rng.normal(size=cols) * 0.3 + (0 if "bias" in k else 1), pst, 0, shift)
    return {k: v[0] for k, v in t.items()}, {k: v[1] for k, v in t.items()}


def f32(n):
    import torch
    return torch.full((n,), 7.0, device="cuda")


def norm_bound(x, xh, rstd, kind, d):
    """Error of a normalised row known to float32 statistics."""
    mean = np.abs(x).mean(1, keepdims=True) if kind == "layer" else 0.0
    return d * U * (2 * np.abs(xh) + mean * rstd[:, None])


NORM_CASES = [("rms", "rms", True, 0.1), ("layer", "layer", True, 0.25), ("none", "rms", False, 0.0), ("rms", "none", True, 0.0),
              ("layer", "rms", False, 1.0), ("none", "layer", True, 0.5)]


@pytest.mark.parametrize("post,pre,gate,p", NORM_CASES)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_blocknorm_forward(nsm, h, rows, cols, types, post, pre, gate, p):
    sst, bst = types
    pad, shift = (3, 1) if cols % 2 else (8, 0)
    pst = "fp32" if rows % 2 else bst
    rng = np.random.default_rng([5, rows, cols])
    t, v = junction(rng, rows, cols, sst, bst, pst, post, pre, gate, True, pad, shift)
    s, y = blank(rows, cols, sst, pad, shift), blank(rows, cols, bst, pad, shift)
    st = {k: f32(rows) for k, on in (("post_mean", post == "layer"), ("post_rstd", post != "none"), ("pre_mean", pre == "layer"),
                                     ("pre_rstd", pre != "none")) if on}
    y8 = act8_blank(nsm, rows, cols, pad, shift) if pre != "none" else None
    alpha, beta, seed, off = 0.75, -0.5, 12345, 678
    x = t.pop("x")
    nsm.muon_blocknorm_forward(h, x, s=s, y=y if pre != "none" else None, post_norm=post, pre_norm=pre, residual_scale=alpha,
                               branch_scale=beta, drop=nsm.Dropout(p, seed, off) if p else None, y8=y8, **t, **st)
    fac = bo.dropout_factors(rows, cols, p, seed, off) if p else np.ones((rows, cols))
    want, pm, pr = bo.junction_stream(v["x"], v["branch"], post, v.get("post_gain"), v.get("post_bias"), v.get("gate"), alpha,
                                      beta, fac)
    d = depth(cols)
    w = np.abs(beta * v.get("post_gain", np.ones(cols)) * v.get("gate", np.ones(cols)))
    b = np.abs(beta * v.get("post_bias", np.zeros(cols)) * v.get("gate", np.ones(cols)))
    oh = v["branch"]
    eo = 0.0
    if post != "none":
        oh = bo.norm(v["branch"], post, 1e-5)[0]
        eo = norm_bound(v["branch"], oh, pr, post, d)
        close(host(st["post_rstd"]), pr, d * U * pr, "post_rstd")
    if post == "layer":
        close(host(st["post_mean"]), pm, d * U * np.abs(v["branch"]).mean(1), "post_mean")
    tol = fac * (eo * w + 8 * U * (np.abs(oh) * w + b)) + 2 * U * (np.abs(alpha * v["x"]) + np.abs(want))
    close(host(s), want, tol + HALF[sst] * np.abs(want), "s")
    assert padding_kept(s)
    if pre == "none":
        return
    sv = host(s)                     # the norm is of the stream as stored
    wy, m, r = bo.junction_norm(sv, pre, v["pre_gain"], v.get("pre_bias"))
    close(host(st["pre_rstd"]), r, d * U * r, "pre_rstd")
    if pre == "layer":
        close(host(st["pre_mean"]), m, d * U * np.abs(sv).mean(1), "pre_mean")
    xh = bo.norm(sv, pre, 1e-5)[0]
    ty = norm_bound(sv, xh, r, pre, d) * np.abs(v["pre_gain"]) + 4 * U * (np.abs(wy) + np.abs(v.get("pre_bias", 0.0)))
    close(host(y), wy, ty + HALF[bst] * np.abs(wy), "y")
    check_act8(y8, wy, ty, "y8")
    assert padding_kept(y) and padding_kept(y8.codes) and padding_kept(y8.exponents)
    # the stream in place gives the same bits
    nsm.muon_blocknorm_forward(h, x, s=x, y=blank(rows, cols, bst, pad, shift), post_norm=post, pre_norm=pre, residual_scale=alpha,
                               branch_scale=beta, drop=nsm.Dropout(p, seed, off) if p else None, **t)
    assert (host(x) == sv).all()


@pytest.mark.parametrize("post,pre,gate,p", NORM_CASES)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_blocknorm_backward(nsm, h, rows, cols, types, post, pre, gate, p):
    sst, bst = types
    pad, shift = (3, 1) if cols % 2 else (8, 0)
    pst = "fp32" if rows % 2 else bst
    rng = np.random.default_rng([6, rows, cols])
    t, v = junction(rng, rows, cols, sst, bst, pst, post, pre, gate, True, pad, shift)
    t.pop("pre_bias", None)
    sv, s = v.pop("x"), t.pop("x")
    acc = rows % 3 == 0
    st, sh = {}, {}
    for k, kind, a in (("post", post, v["branch"]), ("pre", pre, sv)):
        if kind == "none":
            continue
        _, m, r = bo.norm(a, kind, 1e-5)
        st[k + "_rstd"], sh[k + "_rstd"] = dev(r, "fp32")
        if kind == "layer":
            st[k + "_mean"], sh[k + "_mean"] = dev(m, "fp32")
    dy, dyv = dev(rng.normal(size=(rows, cols)), bst, pad, shift)
    ds, dsv = dev(rng.normal(size=(rows, cols)), sst, pad, shift)
    use_ds = pre == "none" or rows % 4 != 3
    dx, db = blank(rows, cols, sst, pad, shift), blank(rows, cols, bst, pad, shift)
    names = [k for k in ("post_gain", "post_bias", "gate", "pre_gain") if k in t] + (["pre_bias"] if pre == "layer" else [])
    g = {"d" + k: dev(rng.normal(size=cols), pst, 0, shift) for k in names}
    old = {k: (x[1] if acc else 0.0) for k, x in g.items()}
    alpha, beta, seed, off = 0.75, -0.5, 54321, 876
    kw = dict(dy=dy if pre != "none" else None, ds=ds if use_ds else None, s=s if pre != "none" else None, dbranch=db,
              post_norm=post, pre_norm=pre, residual_scale=alpha, branch_scale=beta,
              drop=nsm.Dropout(p, seed, off) if p else None, accumulate=acc, **t, **st)
    nsm.muon_blocknorm_backward(h, dx, **kw, **{k: x[0] for k, x in g.items()})
    fac = bo.dropout_factors(rows, cols, p, seed, off) if p else np.ones((rows, cols))
    ds_ = dsv if use_ds else np.zeros_like(sv)
    want = bo.junction_grad(sh, dyv, ds_, sv, v["branch"], post, v.get("post_gain"), v.get("post_bias"), v.get("gate"), pre,
                            v.get("pre_gain"), alpha, beta, fac)
    d, one = depth(cols), np.ones(cols)

    def mean(a):
        return np.abs(a).mean(1, keepdims=True)

    eg = U * np.abs(ds_)
    gr = ds_
    if pre != "none":
        r = sh["pre_rstd"][:, None]
        xh = (sv - sh.get("pre_mean", np.zeros(rows))[:, None]) * r
        a = dyv * v["pre_gain"]
        c1 = mean(a) if pre == "layer" else 0.0
        eg = eg + r * (d * U * (c1 + np.abs(xh) * mean(a * xh)) + 8 * U * (np.abs(a) + c1 + np.abs(xh) * mean(a * xh)))
        gr = want["dx"] / alpha
        close(host(g["dpre_gain"][0]), want["dpre_gain"] + old["dpre_gain"], (rows + 12) * U * np.abs(dyv * xh).sum(0) +
              (2 * U + HALF[pst]) * np.abs(want["dpre_gain"] + old["dpre_gain"]) + U * np.abs(old["dpre_gain"]), "dpre_gain")
        if pre == "layer":
            close(host(g["dpre_bias"][0]), want["dpre_bias"] + old["dpre_bias"], (rows + 12) * U * np.abs(dyv).sum(0) +
                  (2 * U + HALF[pst]) * np.abs(want["dpre_bias"] + old["dpre_bias"]) + U * np.abs(old["dpre_bias"]), "dpre_bias")
    eg = eg + 2 * U * np.abs(gr)
    close(host(dx), want["dx"], alpha * eg + (2 * U + HALF[sst]) * np.abs(want["dx"]), "dx")
    e, ee = np.abs(gr * fac), (eg + U * np.abs(gr)) * fac
    w = np.abs(beta * v.get("post_gain", one) * v.get("gate", one))
    bb, eb = e * w, ee * w + 6 * U * e * w
    oh = v["branch"]
    if post == "none":
        close(host(db), want["dbranch"], eb + HALF[bst] * np.abs(want["dbranch"]), "dbranch")
    else:
        r = sh["post_rstd"][:, None]
        oh = (v["branch"] - sh.get("post_mean", np.zeros(rows))[:, None]) * r
        lay = 1.0 if post == "layer" else 0.0
        ah = np.abs(oh)
        tol = r * (eb + lay * (mean(eb) + d * U * mean(bb)) + ah * (mean(eb * ah) + (d + 6) * U * mean(bb * ah)) +
                   8 * U * (bb + lay * mean(bb) + ah * mean(bb * ah)))
        close(host(db), want["dbranch"], tol + HALF[bst] * np.abs(want["dbranch"]), "dbranch")
    s_tol = (ee * np.abs(oh)).sum(0) + (rows + 16) * U * (e * np.abs(oh)).sum(0)
    d_tol = ee.sum(0) + (rows + 16) * U * e.sum(0)
    gate_, gain_, bias_ = (np.abs(v.get(k, z)) for k, z in (("gate", one), ("post_gain", one), ("post_bias", 0 * one)))
    mags = {"dpost_gain": (abs(beta) * gate_ * s_tol), "dpost_bias": abs(beta) * gate_ * d_tol,
            "dgate": abs(beta) * (gain_ * s_tol + bias_ * d_tol)}
    for k, m in mags.items():
        if k in g:
            x = want[k] + old[k]
            # (dgate is a difference of two terms that may cancel: their own roundings count)
            terms = np.abs(want[k]) if k != "dgate" else abs(beta) * (gain_ * (e * np.abs(oh)).sum(0) + bias_ * e.sum(0))
            close(host(g[k][0]), x, m + 6 * U * terms + (2 * U + HALF[pst]) * np.abs(x) + U * np.abs(old[k]), k)
    assert padding_kept(dx) and padding_kept(db)
    if use_ds:                       # dx over ds: the same bits
        first = host(dx)
        nsm.muon_blocknorm_backward(h, ds, **{**kw, "ds": ds, "dbranch": blank(rows, cols, bst, pad, shift)})
        assert (host(ds) == first).all()


@pytest.mark.parametrize("cols", [40, 1024, 4095, 9000])
def test_blocknorm_without_a_branch_is_a_norm(nsm, h, cols):
    """Against the layer norm's own entry points, and an RMS norm without a gain."""
    import torch
    torch.manual_seed(1)
    x, dy = torch.randn(50, cols, device="cuda").bfloat16(), torch.randn(50, cols, device="cuda").bfloat16()
    g, b = torch.randn(cols, device="cuda").bfloat16(), torch.randn(cols, device="cuda").bfloat16()
    y = [torch.empty_like(x) for _ in range(3)]
    m, r = [f32(50) for _ in range(2)], [f32(50) for _ in range(3)]
    nsm.muon_layernorm_forward(h, x, g, b, y[0], mean=m[0], rstd=r[0])
    nsm.muon_blocknorm_forward(h, x, y=y[1], pre_norm="layer", pre_gain=g, pre_bias=b, pre_mean=m[1], pre_rstd=r[1])
    nsm.muon_blocknorm_forward(h, x, y=y[2], pre_norm="rms", pre_rstd=r[2])
    close(host(y[1]), host(y[0]), 2.0 ** -7 * np.abs(host(y[0])) + 1e-5, "y")      # two roundings to bf16
    close(host(r[1]), host(r[0]), 2 * depth(cols) * U * host(r[0]), "rstd")
    xv = host(x)
    wy, _, wr = bo.junction_norm(xv, "rms")
    close(host(y[2]), wy, 2 * depth(cols) * U * np.abs(wy) + 2.0 ** -8 * np.abs(wy), "rms y")
    dx, dg, db = [torch.empty_like(x) for _ in range(2)], [torch.empty_like(g) for _ in range(2)], [torch.empty_like(g) for _ in range(2)]
    nsm.muon_layernorm_backward(h, dy, x, g, m[0], r[0], dx[0], dg[0], dbias=db[0])
    nsm.muon_blocknorm_backward(h, dx[1], dy=dy, s=x, pre_norm="layer", pre_gain=g, pre_mean=m[0], pre_rstd=r[0], dpre_gain=dg[1],
                                dpre_bias=db[1])
    for a, c in ((dx, "dx"), (dg, "dgain"), (db, "dbias")):
        close(host(a[1]), host(a[0]), 2.0 ** -7 * np.abs(host(a[0])) + 2e-4, c)


def test_blocknorm_constant_and_zero_rows(nsm, h):
    """A layer norm of equal values is its bias whatever their size and place among the
    waves; an RMS norm of zeros is 0; an infinity makes its own row NaN only."""
    import torch
    for cols in (24, 700, 1536, 4100, 9000):
        x = torch.full((6, cols), 1e4 / 3, device="cuda")
        y, b = torch.empty_like(x), torch.randn(cols, device="cuda")
        nsm.muon_blocknorm_forward(h, x, y=y, pre_norm="layer", pre_bias=b)
        assert bool((y == b).all()), cols
        x.zero_()
        x[3, cols // 2] = float("inf")
        nsm.muon_blocknorm_forward(h, x, y=y, pre_norm="rms")
        assert bool((y[[0, 1, 2, 4, 5]] == 0).all()) and bool(torch.isnan(y[3, cols // 2])), cols


@pytest.mark.parametrize("cols", [6, 520, 4095, 9000])
def test_dropped_branch_elements_add_nothing(nsm, h, cols):
    """NaN and infinities where the mask drops: the stream, the branch's gradient and the
    gate's are as if zeros stood there."""
    import torch
    torch.manual_seed(2)
    rows, p = 12, 0.4
    keep = torch.from_numpy(bo.dropout_factors(rows, cols, p, 5, 6) != 0).cuda()
    x, ds, gate = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda"), torch.randn(cols, device="cuda")
    clean = torch.randn(rows, cols, device="cuda") * keep
    bad = torch.where(keep, clean, torch.where(clean.abs().cumsum(1) % 2 > 1, float("nan"), float("inf")))
    out = []
    for b in (clean, bad):
        s, dx, db, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(gate)
        drop = nsm.Dropout(p, 5, 6)
        nsm.muon_blocknorm_forward(h, x, branch=b, s=s, gate=gate, drop=drop)
        nsm.muon_blocknorm_backward(h, dx, ds=ds, branch=b, dbranch=db, gate=gate, dgate=dg, drop=drop)
        out.append((s, dx, db, dg))
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("p", [0.0, 0.4])
@pytest.mark.parametrize("cols", [24, 1000, 9000])
def test_infinite_gradient_beside_a_zero_branch(nsm, h, cols, p):
    """Infinity times 0 is NaN where the element is kept, and nothing where it is dropped."""
    import torch
    torch.manual_seed(3)
    rows = 6
    keep = torch.from_numpy(bo.dropout_factors(rows, cols, p, 7, 8) != 0).cuda()
    ds, branch = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    ds[2, ::3], branch[2, ::3] = float("inf"), 0.0
    gate = torch.ones(cols, device="cuda")
    dx, db, dg = torch.empty_like(ds), torch.empty_like(ds), torch.empty_like(gate)
    nsm.muon_blocknorm_backward(h, dx, ds=ds, branch=branch, dbranch=db, gate=gate, dgate=dg, drop=nsm.Dropout(p, 7, 8))
    want = torch.zeros(cols, dtype=torch.bool, device="cuda")
    want[::3] = keep[2, ::3]
    assert torch.equal(dg.isnan(), want) and not dg.isinf().any()


@pytest.mark.parametrize("cols", [5, 1000, 9000])
def test_blocknorm_backward_of_a_plain_residual(nsm, h, cols):
    """No norms, no gate: the branch itself is not needed, gradients are scaled copies."""
    import torch
    ds = torch.randn(7, cols, device="cuda")
    dx, db = torch.empty_like(ds), torch.empty(7, cols, device="cuda", dtype=torch.bfloat16)
    nsm.muon_blocknorm_backward(h, dx, ds=ds, dbranch=db, residual_scale=0.5, branch_scale=0.25)
    assert torch.equal(dx, ds * 0.5) and torch.equal(db, (ds * 0.25).bfloat16())


def test_blocknorm_rows_far_apart(nsm, h):
    """Rows whose offsets pass 2^31 elements, forward and backward."""
    import torch
    rows, ld = 70000, 32768
    big = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    x, b, s, y, dx, db = (big[:, 64 * k:64 * k + 24] for k in range(6))
    x.normal_()
    b.normal_()
    r = torch.empty(rows, device="cuda")
    nsm.muon_blocknorm_forward(h, x, branch=b, s=s, y=y, pre_norm="rms", pre_rstd=r)
    want = x.float() + b.float()
    close(host(s), host(want), 2.0 ** -8 * np.abs(host(want)), "s")
    sv = host(s)
    xh = sv / np.sqrt((sv ** 2).mean(1, keepdims=True) + 1e-5)
    close(host(y), xh, (2.0 ** -8 + 2 * depth(24) * U) * np.abs(xh), "y")
    nsm.muon_blocknorm_backward(h, dx, dy=x, s=s, dbranch=db, pre_norm="rms", pre_rstd=r)
    g = bo.junction_grad({"pre_rstd": host(r)}, host(x), None, sv, pre="rms")["dx"]
    close(host(dx), g, 2.0 ** -8 * np.abs(g) + 1e-5 * np.abs(host(r))[:, None] * (1 + np.abs(xh)) * np.abs(host(x)).max(), "dx")
    assert torch.equal(dx, db)


def test_two_handles_on_two_streams(nsm, h):
    """Blocks that run at one time on handles of their own give what they give alone."""
    import torch
    h2 = nsm.muon_init(0)
    try:
        a = Block(nsm, h, 700, 512, 1000, "in_out", "silu", 0.1, "rms", "rms", seed=1)
        b = Block(nsm, h2, 650, 480, 904, "out_in", "gelu", 0.2, "layer", "layer", seed=2)
        alone = []
        for x in (a, b):
            x.run()
            torch.cuda.synchronize()
            alone.append(x.outputs())
        s = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(4):
            for x, st in zip((a, b), s):
                st.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(st):
                    x.run()
        torch.cuda.synchronize()
        for x, want in zip((a, b), alone):
            assert all(torch.equal(v, want[k]) for k, v in x.outputs().items())
    finally:
        nsm.muon_destroy(h2)


def test_blocknorm_no_rows(nsm, h):
    import torch
    e = torch.empty(0, 40, device="cuda")
    g, dg, dp = torch.ones(40, device="cuda"), torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    nsm.muon_blocknorm_forward(h, e, branch=e, s=e, y=e, pre_norm="rms", pre_gain=g)
    kw = dict(ds=e, dy=e, s=e, branch=e, dbranch=e, pre_norm="rms", pre_gain=g, pre_rstd=f32(0), gate=g)
    nsm.muon_blocknorm_backward(h, e, dpre_gain=dg, dgate=dp, accumulate=True, **kw)
    assert bool((dg == 3).all()) and bool((dp == 3).all())
    nsm.muon_blocknorm_backward(h, e, dpre_gain=dg, dgate=dp, **kw)
    assert bool((dg == 0).all()) and bool((dp == 0).all())
    w, dw = torch.ones(40, 8, device="cuda"), [torch.full((40, 8), 3.0, device="cuda") for _ in range(2)]
    e8 = torch.empty(0, 8, device="cuda")
    nsm.muon_gated_forward(h, e, w, w, e8, gate_out=nsm.Act8.empty(0, 8), up_out=nsm.Act8.empty(0, 8))
    nsm.muon_gated_grad_hidden(h, e, w.t().contiguous(), e8, e8, e8, e8, h_out=e8)
    nsm.muon_gated_grad_input(h, e8, e8, w, w, e)
    nsm.muon_gated_grad_weight(h, nsm.Act8.empty(0, 40), e8, e8, *dw)
    nsm.muon_dropout(h, e, e, nsm.Dropout(0.5, 1))
    torch.cuda.synchronize()
    assert all(bool((d == 0).all()) for d in dw)


# ---- the operators together ---------------------------------------------------------------

class Block:
    """A feed-forward block on tensors of its own: norm, gated projections, down
    projection, and the junction with dropout behind it; forward and backward."""

    def __init__(self, nsm, h, rows, n, f, lay, act, p, post, pre, step=None, seed=0, eight=True):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf = torch.bfloat16

        def rnd(*s, std=1.0, mean=0.0):
            return torch.empty(*s, device="cuda").normal_(mean, std, generator=g).to(bf)

        def out(*s, dt=bf):
            return torch.empty(*s, device="cuda", dtype=dt)

        w = (lambda i, o: rnd(o, i, std=i ** -0.5)) if lay == "out_in" else (lambda i, o: rnd(i, o, std=i ** -0.5))
        self.nsm, self.h, self.lay, self.act, self.post, self.pre = nsm, h, lay, act, post, pre
        self.drop = nsm.Dropout(p, 99, 7, step=step) if p else None
        self.shape, self.p = (rows, n, f), p
        self.t = t = dict(x=rnd(rows, n), ds=rnd(rows, n, std=0.1), dy=rnd(rows, n, std=0.1), wg=w(n, f), wu=w(n, f), wd=w(f, n),
                          g1=rnd(n, std=0.1, mean=1), g2=rnd(n, std=0.1, mean=1), pg=rnd(n, std=0.1, mean=1) if post != "none" else None,
                          gate=rnd(n, std=0.1, mean=0.5))
        for k, c in (("n1", n), ("h", f), ("o", n), ("s", n), ("y", n), ("do", n), ("h2", f), ("dzg", f), ("dzu", f), ("dn1", n),
                     ("dxr", n), ("dx", n)):
            t[k] = out(rows, c)
        for k in ("r1", "rp", "r2", "m1", "m2", "mp"):
            t[k] = out(rows, dt=torch.float32)
        for k in ("wg", "wu", "wd", "g1", "g2", "pg", "gate"):
            t["d" + k] = torch.empty_like(t[k]) if t[k] is not None else None
        mk = (lambda c: nsm.Act8.empty(rows, c)) if eight else (lambda c: out(rows, c))
        self.n8, self.zg, self.zu = (nsm.Act8.empty(rows, n) if eight else None), mk(f), mk(f)

    def run(self):
        nsm, h, t, lay = self.nsm, self.h, self.t, self.lay
        lm = self.pre == "layer"
        m1, m2 = (t["m1"], t["m2"]) if lm else (None, None)
        rp = t["rp"] if self.post != "none" else None
        j = dict(post_norm=self.post, post_gain=t["pg"], gate=t["gate"], pre_norm=self.pre, pre_gain=t["g2"], branch_scale=0.5,
                 drop=self.drop, post_rstd=rp, post_mean=t["mp"] if self.post == "layer" else None, pre_mean=m2,
                 pre_rstd=t["r2"])
        nsm.muon_blocknorm_forward(h, t["x"], y=t["n1"], pre_norm=self.pre, pre_gain=t["g1"], pre_mean=m1, pre_rstd=t["r1"],
                                   y8=self.n8)
        nsm.muon_gated_forward(h, t["n1"], t["wg"], t["wu"], t["h"], act=self.act, gate_out=self.zg, up_out=self.zu, w_layout=lay)
        nsm.muon_linear_forward(h, t["h"], t["wd"], t["o"], w_layout=lay)
        nsm.muon_blocknorm_forward(h, t["x"], branch=t["o"], s=t["s"], y=t["y"], **j)
        nsm.muon_blocknorm_backward(h, t["dxr"], ds=t["ds"], dy=t["dy"], s=t["s"], branch=t["o"], dbranch=t["do"],
                                    dpost_gain=t["dpg"], dgate=t["dgate"], dpre_gain=t["dg2"], **j)
        nsm.muon_gated_grad_hidden(h, t["do"], t["wd"], self.zg, self.zu, t["dzg"], t["dzu"], act=self.act, h_out=t["h2"],
                                   w_layout=lay)
        nsm.muon_linear_grad_weight(h, t["h2"], t["do"], t["dwd"], w_layout=lay)
        nsm.muon_gated_grad_input(h, t["dzg"], t["dzu"], t["wg"], t["wu"], t["dn1"], w_layout=lay)
        nsm.muon_gated_grad_weight(h, self.n8 if self.n8 is not None else t["n1"], t["dzg"], t["dzu"], t["dwg"], t["dwu"],
                                   w_layout=lay)
        nsm.muon_blocknorm_backward(h, t["dx"], ds=t["dxr"], dy=t["dn1"], s=t["x"], pre_norm=self.pre, pre_gain=t["g1"],
                                    pre_mean=m1, pre_rstd=t["r1"], dpre_gain=t["dg1"])

    OUT = ("s", "y", "dx", "dwg", "dwu", "dwd", "dg1", "dg2", "dpg", "dgate")

    def outputs(self):
        return {k: self.t[k].clone() for k in self.OUT if self.t[k] is not None}

    def oracle(self, offset=7):
        """The exact block: no rounding anywhere."""
        v = {k: host(self.t[k]) for k in ("x", "ds", "dy", "wg", "wu", "wd", "g1", "g2", "pg", "gate") if self.t[k] is not None}
        rows, n, _ = self.shape
        fac = bo.dropout_factors(rows, n, self.p, 99, offset) if self.p else 1.0
        n1, m1, r1 = bo.junction_norm(v["x"], self.pre, v["g1"])
        hh, zg, zu = bo.gated(n1, v["wg"], v["wu"], None, None, self.act, self.lay)
        o = hh @ lo.weight_in_out(v["wd"], self.lay)
        s, pm, pr = bo.junction_stream(v["x"], o, self.post, v.get("pg"), None, v["gate"], 1.0, 0.5, fac)
        y, m2, r2 = bo.junction_norm(s, self.pre, v["g2"])
        st = {k: x for k, x in (("pre_mean", m2), ("pre_rstd", r2), ("post_mean", pm), ("post_rstd", pr)) if x is not None}
        j = bo.junction_grad(st, v["dy"], v["ds"], s, o, self.post, v.get("pg"), None, v["gate"], self.pre, v["g2"], 1.0, 0.5, fac)
        dzg, dzu, _, _ = bo.gated_grad_hidden(j["dbranch"], v["wd"], zg, zu, self.act, self.lay)
        dn1 = bo.gated_grad_input(dzg, dzu, v["wg"], v["wu"], None, self.lay)
        k = bo.junction_grad({"pre_mean": m1, "pre_rstd": r1}, dn1, j["dx"], v["x"], pre=self.pre, pre_gain=v["g1"])
        r = dict(s=s, y=y, dx=k["dx"], dwg=lo.linear_grad_weight(n1, dzg, self.lay)[0], dg1=k["dpre_gain"], dg2=j["dpre_gain"],
                 dwu=lo.linear_grad_weight(n1, dzu, self.lay)[0], dwd=lo.linear_grad_weight(hh, j["dbranch"], self.lay)[0],
                 dgate=j["dgate"])
        return {**r, **({"dpg": j["dpost_gain"]} if self.post != "none" else {})}


@pytest.mark.parametrize("rows,n,f,lay,act,p,post,pre", [(257, 256, 704, "in_out", "silu", 0.1, "rms", "rms"),
                                                         (100, 200, 333, "out_in", "gelu", 0.0, "none", "layer"),
                                                         (1024, 512, 1408, "in_out", "silu", 0.2, "rms", "rms")])
def test_block_against_the_exact_block(nsm, h, rows, n, f, lay, act, p, post, pre):
    """At most twelve roundings lie between the inputs and any output, each at most
    2^-8 (bf16) or 1/127 (a checkpoint) of its value: 12 / 127 in the worst case, and as
    their signs are independent about sqrt(12) / sqrt(3) / 127 = 1.6 % of the norm."""
    b = Block(nsm, h, rows, n, f, lay, act, p, post, pre)
    b.run()
    want = b.oracle()
    for k, got in b.outputs().items():
        e = np.linalg.norm(host(got) - want[k]) / np.linalg.norm(want[k])
        assert e < 0.0235, (k, e)          # one and a half times that


def test_block_is_the_same_every_time_on_any_stream(nsm, h):
    import torch
    b = Block(nsm, h, 300, 320, 520, "in_out", "silu", 0.1, "rms", "rms")
    b.run()
    first = b.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        for k in Block.OUT:
            b.t[k].fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            b.run()
        s.synchronize()
        assert all(torch.equal(v, first[k]) for k, v in b.outputs().items())


def test_captured_block_beside_eager_calls(nsm, h):
    """A captured forward and backward pass with a step counter: replays equal the eager
    block at each step, also after eager calls of larger sizes on the same handle."""
    import torch
    step, count = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    b = Block(nsm, h, 200, 256, 512, "in_out", "silu", 0.1, "rms", "rms", step=step)
    e = Block(nsm, h, 200, 256, 512, "in_out", "silu", 0.1, "rms", "rms", step=count)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.run()
        step.add_(1)
    seen = []
    for n in range(3):
        for k in Block.OUT:
            b.t[k].fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = b.outputs()
        e.run()
        count.add_(1)
        torch.cuda.synchronize()
        assert all(torch.equal(v, got[k]) for k, v in e.outputs().items()), n
        seen.append(got["s"])
        Block(nsm, h, 900 + 300 * n, 333, 777, "out_in", "gelu", 0.0, "none", "rms").run()
        torch.cuda.synchronize()
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_capture_needs_a_resident_workspace(nsm):
    import torch
    hd = nsm.muon_init(0)
    try:
        x, w = torch.randn(64, 100, device="cuda").bfloat16(), torch.randn(100, 60, device="cuda").bfloat16()
        y = torch.empty(64, 60, device="cuda", dtype=torch.bfloat16)     # rows of 120 bytes: operands are re-laid
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            with pytest.raises(nsm.MuonError, match="captured"):
                nsm.muon_gated_forward(hd, x, w, w, y)
            torch.zeros(8, device="cuda").add_(1)
    finally:
        nsm.muon_destroy(hd)


def test_weights_of_one_tensor(nsm, h):
    """Both projections as views of one weight, of either layout, and both gradients
    into one tensor."""
    import torch
    torch.manual_seed(3)
    x = torch.randn(130, 96, device="cuda").bfloat16()
    for lay in ("in_out", "out_in"):
        w = torch.randn(*((96, 160) if lay == "in_out" else (160, 96)), device="cuda").bfloat16()
        a, b = (w[:, :80], w[:, 80:]) if lay == "in_out" else (w[:80], w[80:])
        y = [torch.empty(130, 80, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        nsm.muon_gated_forward(h, x, a, b, y[0], w_layout=lay)
        nsm.muon_gated_forward(h, x, a.contiguous(), b.contiguous(), y[1], w_layout=lay)
        assert torch.equal(*y)
        z = torch.randn(130, 160, device="cuda").bfloat16()
        dz, dw = (z[:, :80], z[:, 80:]), torch.empty_like(w)
        da, db = (dw[:, :80], dw[:, 80:]) if lay == "in_out" else (dw[:80], dw[80:])
        nsm.muon_gated_grad_weight(h, x, *dz, da, db, w_layout=lay)
        want = x.float().t() @ z.float()
        want = want.t() if lay == "out_in" else want
        close(host(dw), host(want), 2.0 ** -8 * np.abs(host(want)) + 1e-3, lay)
