"""GPU parity of the layer operators through the C ABI against the float64
oracle, element by element.

Bounds (u = 2^-24, the float32 unit roundoff; h = half a step of the result's
type relative to it, 2^-8 for bf16 and 2^-24 for float32):

  - a float32 sum of n products is off by at most (n + 8) u times the sum of
    their magnitudes, in any order;
  - layer norm: a row's sums run through at most D = 64 + cols / 512 additions
    one after the other (a lane's elements, the lanes, the waves), so a mean is
    off by D u mean|.|, and rstd by D u relative;
  - an activation adds at most 8 u (1 + |value|), its derivative 16 u (rounding
    of its argument times the logistic's slope, a few units of arithmetic);
  - each output is rounded once: h |result|.
"""

import numpy as np
import pytest

from oracle import decode
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_matrix_step_amd as m
    return m


@pytest.fixture()
def h(nsm):
    hd = nsm.muon_init(0)
    yield hd
    nsm.muon_destroy(hd)


def dev(x, st, ld_pad=0, shift=0):
    """x as a device tensor of storage `st`, rows ld_pad elements apart, starting
    `shift` elements past its allocation; and its exact stored values."""
    import torch
    dt = torch.bfloat16 if st == "bf16" else torch.float32
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dt)
    val = t.double().numpy()
    if t.dim() == 1:
        big = torch.full((t.numel() + shift,), 7.0, dtype=dt, device="cuda")
        big[shift:] = t.cuda()
        return big[shift:], val
    r, c = t.shape
    ld = c + ld_pad
    big = torch.full((r * ld + shift,), 7.0, dtype=dt, device="cuda")
    v = big[shift:].view(r, ld)[:, :c]
    v.copy_(t.cuda())
    return v, val


def blank(r, c, st, ld_pad=0, shift=0):
    import torch
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, "i8": torch.int8, "u8": torch.uint8}[st]
    big = torch.full((r * (c + ld_pad) + shift,), 85, dtype=dt, device="cuda")
    return big[shift:].view(r, c + ld_pad)[:, :c]


def padding_kept(v):
    """The elements between the rows of a blank() view still hold 85."""
    big = v.as_strided((v.shape[0], v.stride(0)), (v.stride(0), 1), v.storage_offset())
    return bool((big[:, v.shape[1]:] == 85).all()) if v.stride(0) > v.shape[1] else True


def host(t):
    return t.detach().double().cpu().numpy()


def close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off, worst "
                           f"{float(np.nanmax(np.abs(got - want) / np.maximum(tol, 1e-300))):.2f} x its bound at "
                           f"{np.argwhere(bad)[0]}")


def act8_blank(nsm, r, c, ld_pad=0, shift=0):
    return nsm.Act8(blank(r, c, "i8", ld_pad, shift), blank(r, -(-c // 32), "u8", min(ld_pad, 1), min(shift, 1)))


def act8_dev(nsm, x, ld_pad=0, shift=0):
    import torch
    q, e = lo.act8_encode(x)
    a = act8_blank(nsm, *x.shape, ld_pad, shift)
    a.codes.copy_(torch.from_numpy(q))
    a.exponents.copy_(torch.from_numpy(e))
    return a, lo.act8_decode(q, e)


def check_act8(a, exact, tol, what):
    """The stored checkpoint of values known to `tol`: exponents those of some
    value in reach, elements within half a step of the exact value."""
    e = a.exponents.cpu().numpy()
    lo_e, hi_e = lo.act8_exponents(np.maximum(np.abs(exact) - tol, 0)), lo.act8_exponents(np.abs(exact) + tol)
    assert np.all((e >= lo_e) & (e <= hi_e)), f"{what}: exponents"
    step = np.exp2(np.repeat(e.astype(np.float64) - 127, 32, axis=1)[:, :exact.shape[1]])
    close(lo.act8_decode(a.codes.cpu().numpy(), e), exact, step / 2 + tol, what)


# ---- layer norm ----------------------------------------------------------------

def depth(cols):
    return 64 + cols / 512


def ln_inputs(rows, cols, st, pst, pad=0, shift=0, seed=0):
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))) + 0.5
    return (dev(x, st, pad, shift), dev(1 + 0.1 * rng.standard_normal(cols), pst, 0, shift),
            dev(0.1 * rng.standard_normal(cols), pst, 0, shift))


def ln_tol(xv, gv, bv, mean, rstd, y, st):
    xh = np.abs(xv - mean[:, None]) * rstd[:, None]
    mag = np.abs(xv).mean(1, keepdims=True)
    return (2 * depth(xv.shape[1]) * U * (np.abs(gv) * (xh + rstd[:, None] * mag) + np.abs(bv)) +
            4 * U * np.abs(y) + HALF[st] * np.abs(y))


LN_SHAPES = [(1, 1), (1, 768), (3, 2), (7, 33), (5, 512), (9, 520), (4, 1000), (33, 1024), (6, 1408), (5, 2048),
             (4, 2050), (3, 4096), (3, 5000), (2, 8192), (2, 12288), (2, 16384), (2, 16392), (1, 40001), (700, 96)]


@pytest.mark.parametrize("st,pst", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", LN_SHAPES)
def test_layernorm_forward(nsm, h, rows, cols, st, pst):
    import torch
    for pad, shift in ((0, 0), (8, 0), (3, 1)):
        (x, xv), (g, gv), (b, bv) = ln_inputs(rows, cols, st, pst, pad, shift)
        y = blank(rows, cols, st, pad, shift)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        q = act8_blank(nsm, rows, cols, pad, shift)
        nsm.muon_layernorm_forward(h, x, g, b, y, mean=mean, rstd=rstd, eps=1e-5, y8=q)
        ry, rm, rr = lo.layernorm(xv, gv, bv, float(np.float32(1e-5)))
        tol = ln_tol(xv, gv, bv, rm, rr, ry, st)
        close(host(y), ry, tol, "y")
        close(host(mean), rm, depth(cols) * U * np.abs(xv).mean(1) + U * np.abs(rm), "mean")
        # the variance is off by D u relative from its sum and by the mean's error squared
        dm = (depth(cols) * U * np.abs(xv).mean(1)) ** 2 * rr ** 2
        close(host(rstd), rr, (depth(cols) * U + dm) * rr, "rstd")
        check_act8(q, ry, tol - HALF[st] * np.abs(ry), "y8")
        assert padding_kept(y) and padding_kept(q.codes) and padding_kept(q.exponents)
        nsm.muon_layernorm_forward(h, x, g, None, y, eps=1e-5)     # nothing optional
        r0 = lo.layernorm(xv, gv, None, float(np.float32(1e-5)))[0]
        close(host(y), r0, ln_tol(xv, gv, 0 * bv, rm, rr, r0, st), "y without bias")


@pytest.mark.parametrize("st,pst", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,cols", LN_SHAPES + [(2300, 200)])
def test_layernorm_backward(nsm, h, rows, cols, st, pst):
    import torch
    for pad, shift, add_kind in ((0, 0, "own"), (8, 0, "dx"), (3, 1, None)):
        (x, xv), (g, gv), _ = ln_inputs(rows, cols, st, pst, pad, shift)
        rng = np.random.default_rng([7, rows, cols])
        dy, dyv = dev(rng.standard_normal((rows, cols)), st, pad, shift)
        _, rm, rr = lo.layernorm(xv, gv, None, 1e-5)
        mean, mv = dev(rm, "fp32")
        rstd, rv = dev(rr, "fp32")
        dx, add, av = blank(rows, cols, st, pad, shift), None, 0.0
        if add_kind:
            t, av = dev(rng.standard_normal((rows, cols)), st, pad, shift)
            add = dx if add_kind == "dx" else t
            if add_kind == "dx":
                dx.copy_(t)
        dg0, dg0v = dev(rng.standard_normal(cols), pst, 0, shift)
        db0, db0v = dev(rng.standard_normal(cols), pst, 0, shift)
        acc = add_kind == "dx"
        nsm.muon_layernorm_backward(h, dy, x, g, mean, rstd, dx, dg0, dbias=db0, add=add, accumulate=acc)
        rdx, rdg, rdb = lo.layernorm_grad(dyv, xv, gv, mv, rv, None if add is None else av)
        if acc:
            rdg, rdb = rdg + dg0v, rdb + db0v
        xh, a = (xv - mv[:, None]) * rv[:, None], dyv * gv
        d = depth(cols) * U
        tol = (2 * d * rv[:, None] * (np.abs(a) + np.abs(a).mean(1, keepdims=True) +
                                      np.abs(xh) * np.abs(a * xh).mean(1, keepdims=True)) +
               4 * U * (np.abs(rdx) + np.abs(av)) + HALF[st] * np.abs(rdx))
        close(host(dx), rdx, tol, "dx")
        n = rows + 64
        close(host(dg0), rdg, n * U * np.abs(dyv * xh).sum(0) + (U + HALF[pst]) * np.abs(rdg) + U * np.abs(dg0v), "dgain")
        close(host(db0), rdb, n * U * np.abs(dyv).sum(0) + (U + HALF[pst]) * np.abs(rdb) + U * np.abs(db0v), "dbias")
        assert padding_kept(dx)
        if not acc:   # without dbias the others do not change
            dg1, dx1 = torch.empty_like(dg0), blank(rows, cols, st, pad, shift)
            nsm.muon_layernorm_backward(h, dy, x, g, mean, rstd, dx1, dg1, add=add if add is not dx else None)
            assert torch.equal(dg1, dg0) and torch.equal(dx1, dx)


def test_layernorm_no_rows(nsm, h):
    import torch
    e = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(40, device="cuda")
    v = torch.empty(0, device="cuda")
    nsm.muon_layernorm_forward(h, e, g, None, torch.empty_like(e))
    dg, db = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 4.0, device="cuda")
    nsm.muon_layernorm_backward(h, e, e, g, v, v, torch.empty_like(e), dg, dbias=db, accumulate=True)
    assert bool((dg == 3).all()) and bool((db == 4).all())
    nsm.muon_layernorm_backward(h, e, e, g, v, v, torch.empty_like(e), dg, dbias=db)
    assert bool((dg == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("cols", [96, 1000, 4096, 17000])
def test_layernorm_nan_stays_in_its_row(nsm, h, cols):
    """A NaN or an infinity makes its own row NaN (and its checkpoint's groups);
    a constant row gives the bias."""
    import torch
    (x, xv), (g, gv), (b, bv) = ln_inputs(6, cols, "bf16", "bf16")
    x[1, 5] = float("nan")
    x[3, cols - 1] = float("inf")
    x[4] = 3.0
    y, q = blank(6, cols, "bf16"), act8_blank(nsm, 6, cols)
    nsm.muon_layernorm_forward(h, x, g, b, y, y8=q)
    y, yd = host(y), lo.act8_decode(q.codes.cpu().numpy(), q.exponents.cpu().numpy())
    assert np.isnan(y[[1, 3]]).all() and np.isfinite(y[[0, 2, 4, 5]]).all()
    assert np.isnan(yd[[1, 3]]).all() and np.isfinite(yd[[0, 2, 4, 5]]).all()
    assert np.abs(y[4] - bv).max() <= 1e-6


# ---- 8-bit checkpoints ----------------------------------------------------------

@pytest.mark.parametrize("st", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (4, 32), (5, 33), (64, 1000), (7, 4096), (3, 20000), (1000, 40)])
def test_act8_round_trip_is_exact(nsm, h, rows, cols, st):
    """Codes and exponents equal the oracle's bit for bit; decoding is exact in
    both types."""
    rng = np.random.default_rng([11, rows, cols])
    x = rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-60, 60, (rows, 1)))
    x[:, ::7] = np.exp2(rng.integers(-40, 40, x[:, ::7].shape))      # many ties
    x[0, 0] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2] = 2.0 ** -130 * rng.integers(-3, 4, cols)                # below the smallest step
    for pad, shift in ((0, 0), (8, 0), (5, 3)):
        t, v = dev(x, st, pad, shift)
        q, y = act8_blank(nsm, rows, cols, pad, shift), blank(rows, cols, st, pad, shift)
        nsm.muon_act_encode(h, t, q)
        rq, re = lo.act8_encode(v)
        assert np.array_equal(q.exponents.cpu().numpy(), re)
        assert np.array_equal(q.codes.cpu().numpy(), rq)
        nsm.muon_act_decode(h, q, y)
        assert np.array_equal(host(y), lo.act8_decode(rq, re))
        assert padding_kept(y) and padding_kept(q.codes) and padding_kept(q.exponents)


def test_act8_non_finite_groups(nsm, h):
    import torch
    x = torch.randn(4, 100, device="cuda")
    x[0, 3], x[1, 40], x[2, 99], x[3, 64] = float("nan"), float("inf"), float("-inf"), 3.0e38
    q, y = nsm.Act8.empty(4, 100), torch.empty_like(x)
    nsm.muon_act_encode(h, x, q)
    nsm.muon_act_decode(h, q, y)
    bad = torch.zeros(4, 100, dtype=torch.bool, device="cuda")
    bad[0, :32] = bad[1, 32:64] = bad[2, 96:] = True
    assert torch.equal(torch.isnan(y), bad)
    assert abs(float(y[3, 64]) / 3.0e38 - 1) < 2 ** -7
    rq, re = lo.act8_encode(x.double().cpu().numpy())
    assert np.array_equal(q.exponents.cpu().numpy(), re) and np.array_equal(q.codes.cpu().numpy(), rq)


# ---- the linear layer -------------------------------------------------------------

def lin_tol(k, mag, act_mag, y, st):
    """A product's sum, then an activation of slope at most `act_mag`."""
    return (k + 16) * U * mag * act_mag + 4 * U * np.abs(y) + HALF[st] * np.abs(y)


LIN_SHAPES = [(1, 1, 1), (1, 64, 8), (1, 1024, 384), (2, 40, 72), (16, 256, 128), (17, 100, 50), (64, 512, 512),
              (127, 129, 131), (128, 128, 128), (130, 200, 264), (255, 72, 520), (300, 768, 768), (513, 1408, 264),
              (40, 4096, 136), (1, 333, 999), (900, 1001, 1031), (16, 2051, 776)]


def act_slope(z, kind):
    """Largest slope of the activation near z."""
    return {"none": 1.0, "gelu": 1.2}[kind] if kind != "relu_sq" else 2 * np.abs(z) + 1e-2


@pytest.mark.parametrize("st", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,k,n", LIN_SHAPES)
def test_linear_forward(nsm, h, rows, k, n, layout, st):
    rng = np.random.default_rng([21, rows, k, n])
    x0 = rng.standard_normal((rows, k))
    w0 = rng.standard_normal((n, k) if layout == "out_in" else (k, n)) / np.sqrt(k)
    for pad, shift, act, bst, res_kind, zk in ((0, 0, "gelu", st, None, "act8"), (8, 0, "none", "fp32", "y", "full"),
                                               (3, 1, "relu_sq", "bf16", "own", "act8"), (0, 0, "none", None, None, None)):
        x, xv = dev(x0, st, pad, shift)
        w, wv = dev(w0, st, pad, shift)
        b, bv = dev(rng.standard_normal(n), bst, 0, shift) if bst else (None, np.zeros(n))
        y, res, rv = blank(rows, n, st, pad, shift), None, 0.0
        if res_kind:
            t, rv = dev(rng.standard_normal((rows, n)), st, pad, shift)
            res = t
            if res_kind == "y":
                y.copy_(t)
                res = y
        z = {"act8": lambda: act8_blank(nsm, rows, n, pad, shift), "full": lambda: blank(rows, n, st, pad, shift),
             None: lambda: None}[zk]()
        nsm.muon_linear_forward(h, x, w, y, bias=b, act=act, residual=res, z_out=z, w_layout=layout)
        ry, rz = lo.linear(xv, wv, bv, act, None if res is None else rv, layout)
        mag = np.abs(xv) @ np.abs(lo.weight_in_out(wv, layout)) + np.abs(bv)
        slope = act_slope(rz, act)
        tol = lin_tol(k, mag, slope, ry, st) + 8 * U * (1 + np.abs(ry)) + 2 * U * np.abs(rv)
        close(host(y), ry, tol, f"y ({act}, pad {pad})")
        if zk == "full":
            close(host(z), rz, lin_tol(k, mag, 1.0, rz, st), "z")
            assert padding_kept(z)
        elif zk == "act8":
            check_act8(z, rz, (k + 16) * U * mag, "z8")
            assert padding_kept(z.codes) and padding_kept(z.exponents)
        assert padding_kept(y)


@pytest.mark.parametrize("st", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,k,n", LIN_SHAPES)
def test_linear_grad_input(nsm, h, rows, k, n, layout, st):
    rng = np.random.default_rng([22, rows, k, n])
    dy0 = rng.standard_normal((rows, n))
    w0 = rng.standard_normal((n, k) if layout == "out_in" else (k, n)) / np.sqrt(n)
    for pad, shift, act, zk, add_kind, want_v in ((0, 0, "gelu", "act8", None, True), (8, 0, "relu_sq", "full", "dx", True),
                                                  (3, 1, "gelu", "act8", "own", False), (0, 0, "none", None, None, False)):
        dy, dyv = dev(dy0, st, pad, shift)
        w, wv = dev(w0, st, pad, shift)
        z, zv = None, None
        z0 = rng.standard_normal((rows, k)) * 3
        if zk == "act8":
            z, zv = act8_dev(nsm, z0, pad, shift)
        elif zk == "full":
            z, zv = dev(z0, st, pad, shift)
        dx, add, av = blank(rows, k, st, pad, shift), None, 0.0
        if add_kind:
            t, av = dev(rng.standard_normal((rows, k)), st, pad, shift)
            add = t
            if add_kind == "dx":
                dx.copy_(t)
                add = dx
        v = blank(rows, k, st, pad, shift) if want_v else None
        nsm.muon_linear_grad_input(h, dy, w, dx, act=act, z=z, act_out=v, add=add, w_layout=layout)
        rdx, rv = lo.linear_grad_input(dyv, wv, act, zv, None if add is None else av, layout)
        prod = dyv @ lo.weight_in_out(wv, layout).T
        mag = np.abs(dyv) @ np.abs(lo.weight_in_out(wv, layout)).T
        der = np.abs(lo.activation(zv, act)[1]) if zv is not None else 1.0
        tol = (lin_tol(n, mag, der, rdx, st) + 16 * U * np.abs(prod) * (1 + (der if act == "relu_sq" else 0)) +
               2 * U * np.abs(av))
        close(host(dx), rdx, tol, f"dx ({act}, pad {pad})")
        if want_v:
            close(host(v), rv, 8 * U * (1 + np.abs(rv)) + HALF[st] * np.abs(rv), "act_out")
            assert padding_kept(v)
        assert padding_kept(dx)


@pytest.mark.parametrize("rows,k,n,layout", [(2101, 4096, 40, "in_out"), (2048, 4224, 64, "out_in")])
def test_linear_grad_input_large_outputs(nsm, h, rows, k, n, layout):
    """dx and act(z) together larger than the caches they are kept in."""
    rng = np.random.default_rng([28, rows, k, n])
    dy, dyv = dev(rng.standard_normal((rows, n)), "bf16")
    w, wv = dev(rng.standard_normal((n, k) if layout == "out_in" else (k, n)) / np.sqrt(n), "bf16")
    z, zv = act8_dev(nsm, rng.standard_normal((rows, k)) * 3)
    dx, v = blank(rows, k, "bf16"), blank(rows, k, "bf16")
    nsm.muon_linear_grad_input(h, dy, w, dx, act="gelu", z=z, act_out=v, w_layout=layout)
    rdx, rv = lo.linear_grad_input(dyv, wv, "gelu", zv, None, layout)
    wio = lo.weight_in_out(wv, layout).T
    der = np.abs(lo.activation(zv, "gelu")[1])
    tol = lin_tol(n, np.abs(dyv) @ np.abs(wio), der, rdx, "bf16") + 16 * U * np.abs(dyv @ wio)
    close(host(dx), rdx, tol, "dx")
    close(host(v), rv, 8 * U * (1 + np.abs(rv)) + HALF["bf16"] * np.abs(rv), "act_out")


DW_SHAPES = [(1, 1, 1), (1, 8, 16), (5, 40, 72), (33, 131, 67), (64, 128, 128), (100, 200, 264), (257, 256, 136),
             (1000, 96, 520), (4100, 72, 40), (513, 1408, 264), (1300, 1001, 771)]


@pytest.mark.parametrize("st", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,k,n", DW_SHAPES)
def test_linear_grad_weight(nsm, h, rows, k, n, layout, st):
    rng = np.random.default_rng([23, rows, k, n])
    x0, dy0 = rng.standard_normal((rows, k)), rng.standard_normal((rows, n))
    for pad, shift, xk, dst, bst, acc in ((0, 0, "act8", st, st, False), (8, 0, "full", "fp32", "fp32", True),
                                          (3, 1, "act8", "fp32", "bf16", True), (0, 0, "full", st, None, False),
                                          (3, 1, "full", "bf16", st, False), (8, 0, "act8", st, None, False)):
        x, xv = act8_dev(nsm, x0, pad, shift) if xk == "act8" else dev(x0, st, pad, shift)
        dy, dyv = dev(dy0, st, pad, shift)
        shape = (n, k) if layout == "out_in" else (k, n)
        dw, wv = blank(*shape, dst, pad, shift), 0.0
        if acc:
            t, wv = dev(rng.standard_normal(shape), dst, pad, shift)
            dw.copy_(t)
        db, bv = dev(rng.standard_normal(n), bst, 0, shift) if bst else (None, 0.0)
        nsm.muon_linear_grad_weight(h, x, dy, dw, db=db, accumulate=acc, w_layout=layout)
        rdw, rdb = lo.linear_grad_weight(xv, dyv, layout)
        mag = lo.linear_grad_weight(np.abs(xv), np.abs(dyv), layout)[0]
        if acc:
            rdw, rdb = rdw + wv, rdb + bv
        close(host(dw), rdw, lin_tol(rows, mag, 1.0, rdw, dst) + 2 * U * np.abs(wv), f"dw ({xk}, pad {pad})")
        if bst:
            close(host(db), rdb, (rows + 16) * U * np.abs(dyv).sum(0) + (2 * U + HALF[bst]) * np.abs(rdb) +
                  2 * U * np.abs(bv), "db")
        assert padding_kept(dw)


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,k,n", [(2050, 2048, 1408), (4090, 1024, 4104), (8192, 1000, 2048), (3000, 2051, 1999)])
def test_linear_large_products(nsm, h, rows, k, n, layout):
    """Sizes that take the wider tiles, splits and re-laid operands (ragged rows
    and columns, odd leading dimensions), bf16, against float64 products on the
    GPU; the bounds as above."""
    import torch
    bf = torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + k)

    def rnd(*s, std=1.0):
        return torch.empty(*s, device="cuda").normal_(0, std, generator=g).to(bf)

    def near(got, want, tol, what):
        bad = (got.double() - want).abs() > tol
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"

    def decoded(q):
        step = torch.exp2(q.exponents.double() - 127)
        return q.codes.double() * step.repeat_interleave(32, dim=1)[:, :q.codes.shape[1]]

    x, b, res, dy = rnd(rows, k), rnd(n), rnd(rows, n), rnd(rows, n)
    w = rnd(*((n, k) if layout == "out_in" else (k, n)), std=k ** -0.5)
    wio = (w.t() if layout == "out_in" else w).double()
    y, z8 = torch.empty_like(res), nsm.Act8.empty(rows, n)
    nsm.muon_linear_forward(h, x, w, y, bias=b, act="gelu", residual=res, z_out=z8, w_layout=layout)
    z = x.double() @ wio + b.double()
    mag = x.double().abs() @ wio.abs() + b.double().abs()
    ry = torch.nn.functional.gelu(z, approximate="tanh") + res.double()
    near(y, ry, (k + 16) * U * 1.2 * mag + 8 * U * (1 + ry.abs()) + 2 * U * res.double().abs() + (4 * U + 2.0 ** -8) * ry.abs(), "y")
    step = torch.exp2(z8.exponents.double() - 127).repeat_interleave(32, dim=1)[:, :n]
    near(decoded(z8), z, step / 2 + (k + 16) * U * mag, "z8")
    # through the activation of this layer's own pre-activation sizes: z is rows x k
    zi = nsm.Act8.empty(rows, k)
    nsm.muon_act_encode(h, x, zi)
    dx, v = torch.empty_like(x), torch.empty_like(x)
    nsm.muon_linear_grad_input(h, dy, w, dx, act="relu_sq", z=zi, act_out=v, w_layout=layout)
    zd = decoded(zi).clamp_min(0)
    rdx = (dy.double() @ wio.t()) * 2 * zd
    near(dx, rdx, (n + 16) * U * (dy.double().abs() @ wio.abs().t()) * 2 * zd + (32 * U + 2.0 ** -8) * rdx.abs(), "dx")
    near(v, zd * zd, (4 * U + 2.0 ** -8) * zd * zd, "act_out")
    for xin, xv, dt in ((x, x.double(), bf), (zi, decoded(zi), torch.float32)):
        dw, db = torch.empty(w.shape, device="cuda", dtype=dt), torch.empty(n, device="cuda")
        nsm.muon_linear_grad_weight(h, xin, dy, dw, db=db, w_layout=layout)
        rdw, m = xv.t() @ dy.double(), xv.abs().t() @ dy.double().abs()
        got = dw.t() if layout == "out_in" else dw
        near(got, rdw, (rows + 16) * U * m + (4 * U + (2.0 ** -8 if dt is bf else 2.0 ** -24)) * rdw.abs(), "dw")
        near(db, dy.double().sum(0), (rows + 16) * U * dy.double().abs().sum(0), "db")


def test_linear_no_rows(nsm, h):
    import torch
    bf = torch.bfloat16
    x, dy = torch.empty(0, 40, device="cuda", dtype=bf), torch.empty(0, 72, device="cuda", dtype=bf)
    w, dw = torch.ones(40, 72, device="cuda", dtype=bf), torch.full((40, 72), 3.0, device="cuda", dtype=bf)
    db = torch.full((72,), 2.0, device="cuda")
    nsm.muon_linear_forward(h, x, w, torch.empty(0, 72, device="cuda", dtype=bf))
    nsm.muon_linear_grad_input(h, dy, w, torch.empty(0, 40, device="cuda", dtype=bf))
    nsm.muon_linear_grad_weight(h, x, dy, dw, db=db, accumulate=True)
    assert bool((dw == 3).all()) and bool((db == 2).all())
    nsm.muon_linear_grad_weight(h, x, dy, dw, db=db)
    assert not dw.any() and not db.any()
    nsm.muon_linear_grad_weight(h, nsm.Act8.empty(0, 40), dy, dw, db=db)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("layout", ["in_out", "out_in"])
@pytest.mark.parametrize("rows,k,n", [(200, 136, 264), (200, 133, 267), (300, 72, 128)])
def test_linear_non_finite_operands(nsm, h, rows, k, n, layout):
    """A NaN or an infinity reaches the outputs it takes part in and no others:
    the parts of a tile past the operands' ends contribute nothing, whatever
    the neighbouring memory holds (here NaN)."""
    import torch
    bf = torch.bfloat16

    def nan_around(r, c):
        big = torch.full((r + 2, c + 8), float("nan"), device="cuda", dtype=bf)
        v = big[1:r + 1, :c]
        v.copy_(torch.randn(r, c, device="cuda"))
        return v

    x, w = nan_around(rows, k), nan_around(*((n, k) if layout == "out_in" else (k, n)))
    y = torch.empty(rows, n, device="cuda", dtype=bf)
    nsm.muon_linear_forward(h, x, w, y, w_layout=layout)
    assert bool(torch.isfinite(y).all())
    dy, dx, dw, db = nan_around(rows, n), torch.empty(rows, k, device="cuda", dtype=bf), torch.empty_like(w), \
        torch.empty(n, device="cuda")
    nsm.muon_linear_grad_input(h, dy, w, dx, w_layout=layout)
    nsm.muon_linear_grad_weight(h, x, dy, dw, db=db, w_layout=layout)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all()) and bool(torch.isfinite(db).all())
    x[3, 7] = float("nan")
    nsm.muon_linear_forward(h, x, w, y, w_layout=layout)
    nsm.muon_linear_grad_weight(h, x, dy, dw, w_layout=layout)
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isfinite(torch.cat([y[:3], y[4:]])).all())
    g = dw if layout == "in_out" else dw.t()
    assert bool(torch.isnan(g[7]).all()) and bool(torch.isfinite(torch.cat([g[:7], g[8:]])).all())


@pytest.mark.parametrize("act", ["gelu", "relu_sq"])
def test_activation_over_its_range(nsm, h, act):
    """act and act' from the smallest to the largest pre-activations, through
    the epilogue: dx = 1 * act'(z), act_out = act(z)."""
    import torch
    z0 = np.concatenate([np.linspace(-30, 30, 4001), [0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 9.0, -9.0, 1e18, -1e18]])
    rows, k = z0.size, 8
    z, zv = dev(np.repeat(z0[:, None], k, 1), "fp32")
    dy, w = torch.ones(rows, 1, device="cuda"), torch.ones(k, 1, device="cuda")
    dx, v = torch.empty(rows, k, device="cuda"), torch.empty(rows, k, device="cuda")
    nsm.muon_linear_grad_input(h, dy, w, dx, act=act, z=z, act_out=v)
    with np.errstate(over="ignore", invalid="ignore"):
        rv, rd = lo.activation(zv, act)
    rv, rd = np.where(np.abs(zv) > 1e17, np.where(zv > 0, zv if act == "gelu" else zv * zv, 0.0), rv), \
        np.where(np.abs(zv) > 1e17, np.where(zv > 0, 1.0 if act == "gelu" else 2 * zv, 0.0), rd)
    close(host(v), rv, 8 * U * (1 + np.abs(rv)), "act")
    close(host(dx), rd, 16 * U * (1 + np.abs(rd)), "act'")
    z[0] = float("nan")
    nsm.muon_linear_grad_input(h, dy, w, dx, act=act, z=z, act_out=v)
    assert bool(torch.isnan(dx[0]).all()) and bool(torch.isnan(v[0]).all())


# ---- used together ------------------------------------------------------------------

def _block(nsm, h, t, act, layout, stream=None):
    """One pre-norm block's training pass on the tensors of dict t."""
    x8, z8 = nsm.Act8(*t["xn8"]), nsm.Act8(*t["z8"])
    kw = dict(stream=stream)
    nsm.muon_layernorm_forward(h, t["x"], t["gain"], t["beta"], t["xn"], mean=t["mean"], rstd=t["rstd"], y8=x8, **kw)
    nsm.muon_linear_forward(h, t["xn"], t["w1"], t["h"], bias=t["b1"], act=act, z_out=z8, w_layout=layout, **kw)
    nsm.muon_linear_forward(h, t["h"], t["w2"], t["y"], bias=t["b2"], residual=t["x"], w_layout=layout, **kw)
    nsm.muon_linear_grad_input(h, t["dy"], t["w2"], t["dz"], act=act, z=z8, act_out=t["h2"], w_layout=layout, **kw)
    nsm.muon_linear_grad_weight(h, t["h2"], t["dy"], t["dw2"], db=t["db2"], w_layout=layout, **kw)
    nsm.muon_linear_grad_input(h, t["dz"], t["w1"], t["dxn"], w_layout=layout, **kw)
    nsm.muon_linear_grad_weight(h, x8, t["dz"], t["dw1"], db=t["db1"], w_layout=layout, **kw)
    nsm.muon_layernorm_backward(h, t["dxn"], t["x"], t["gain"], t["mean"], t["rstd"], t["dx"], t["dgain"],
                                dbias=t["dbeta"], add=t["dy"], **kw)


OUTS = ("xn", "h", "y", "dz", "h2", "dw2", "db2", "dxn", "dw1", "db1", "dx", "dgain", "dbeta")


def _block_tensors(rows, d, f, layout, seed=0, dtype=None):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = dtype or torch.bfloat16

    def rnd(*s, std=1.0, mean=0.0):
        return torch.empty(*s, device="cuda").normal_(mean, std, generator=g).to(dtype)

    w1, w2 = ((f, d), (d, f)) if layout == "out_in" else ((d, f), (f, d))
    t = {"x": rnd(rows, d), "dy": rnd(rows, d, std=1e-2), "gain": rnd(d, std=0.1, mean=1.0), "beta": rnd(d, std=0.1),
         "w1": rnd(*w1, std=d ** -0.5), "w2": rnd(*w2, std=f ** -0.5), "b1": rnd(f, std=0.1), "b2": rnd(d, std=0.1)}
    for k, s in {"xn": (rows, d), "h": (rows, f), "y": (rows, d), "dz": (rows, f), "h2": (rows, f), "dxn": (rows, d),
                 "dx": (rows, d), "dw1": w1, "dw2": w2, "db1": (f,), "db2": (d,), "dgain": (d,), "dbeta": (d,)}.items():
        t[k] = torch.full(s, 9.0, device="cuda", dtype=dtype)
    t["mean"], t["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for k, c in (("xn8", d), ("z8", f)):
        t[k] = (torch.empty(rows, c, device="cuda", dtype=torch.int8),
                torch.empty(rows, -(-c // 32), device="cuda", dtype=torch.uint8))
    return t


@pytest.mark.parametrize("act,layout", [("gelu", "in_out"), ("relu_sq", "out_in")])
def test_block_gradients_and_steps(nsm, h, act, layout):
    """A block's forward and backward pass against the float64 gradient of the
    whole block (no 8-bit checkpoints, no roundings in it), then the optimizer
    steps on the gradients.  A gradient element is a sum over independent
    roundings of 2^-9 (bf16 activations) and of at most 2^-7 of a group's
    largest element (8-bit checkpoints, a uniform error of half that at most:
    under 0.012 of the rms for normal values), so a whole gradient's relative
    error stays below 0.03; a wrong term (a missing transpose, factor or
    activation derivative) gives an error of order 1."""
    import torch
    rows, d, f = 333, 256, 640
    t = _block_tensors(rows, d, f, layout, seed=3)
    _block(nsm, h, t, act, layout)
    v = {k: t[k].double().cpu().requires_grad_() for k in ("x", "gain", "beta", "w1", "b1", "w2", "b2")}
    mu = v["x"].mean(1, keepdim=True)
    xn = (v["x"] - mu) / ((v["x"] - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * v["gain"] + v["beta"]
    z = xn @ (v["w1"].t() if layout == "out_in" else v["w1"]) + v["b1"]
    a = torch.nn.functional.gelu(z, approximate="tanh") if act == "gelu" else z.clamp_min(0).square()
    y = a @ (v["w2"].t() if layout == "out_in" else v["w2"]) + v["b2"] + v["x"]
    y.backward(t["dy"].double().cpu())
    want = {"y": y.detach(), "dx": v["x"].grad, "dgain": v["gain"].grad, "dbeta": v["beta"].grad, "dw1": v["w1"].grad,
            "db1": v["b1"].grad, "dw2": v["w2"].grad, "db2": v["b2"].grad}
    for k, r in want.items():
        e = float((t[k].double().cpu() - r).norm() / r.norm())
        print(f"  {k}: relative error {e:.2e}", flush=True)
        assert e < 0.03, (k, e)
    m1, m2 = torch.zeros(t["w1"].shape, device="cuda"), torch.zeros(t["w2"].shape, device="cuda")
    w_old = t["w1"].clone()
    nsm.muon_step(h, [t["w1"], t["w2"]], [t["dw1"], t["dw2"]], [m1, m2], nsm.Hparams())
    vec = ["gain", "beta", "b1", "b2"]
    mom = [torch.zeros(t[k].shape, device="cuda") for k in vec]
    sec = [torch.zeros(t[k].shape, device="cuda") for k in vec]
    nsm.muon_adamw_step(h, [t[k] for k in vec], [t[k] for k in ("dgain", "dbeta", "db1", "db2")], mom, sec,
                        nsm.AdamWHparams())
    torch.cuda.synchronize()
    assert torch.equal(m1, t["dw1"].float()) and not torch.equal(w_old, t["w1"])
    for k in ("w1", "w2", *vec):
        assert bool(torch.isfinite(t[k]).all())


def test_block_same_bits_on_every_call_and_stream(nsm, h):
    import torch
    a, b = _block_tensors(200, 128, 520, "in_out", 5), _block_tensors(200, 128, 520, "in_out", 5)
    _block(nsm, h, a, "gelu", "in_out")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in (_block_tensors(64, 1408, 264, "out_in", 6), b):    # another shape in between, then the same call
        with torch.cuda.stream(s):
            _block(nsm, h, t, "gelu", "in_out" if t is b else "out_in")
    _block(nsm, h, a, "gelu", "in_out", stream=s)                 # the stream given by argument
    torch.cuda.synchronize()
    for k in OUTS:
        assert torch.equal(a[k], b[k]), k


def test_block_captured_into_a_graph(nsm, h):
    """Two shapes captured into two graphs that share the handle's workspaces;
    replayed several times with new inputs and eager calls of larger shapes
    between the replays, every replay equal to the eager result."""
    import torch
    shapes = [(100, 128, 264), (257, 520, 136)]
    ts = [_block_tensors(*s, "in_out", 8) for s in shapes]
    graphs = []
    for t in ts:
        _block(nsm, h, t, "gelu", "in_out")
    torch.cuda.synchronize()
    for t in ts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _block(nsm, h, t, "gelu", "in_out")
        graphs.append(g)
    for rep in range(4):
        big = _block_tensors(600 + 300 * rep, 1032, 2048, "out_in", 20 + rep)
        _block(nsm, h, big, "relu_sq", "out_in")          # grows the workspaces
        for i, (t, g) in enumerate(zip(ts, graphs)):
            new = _block_tensors(*shapes[i], "in_out", 100 + 10 * rep + i)
            for k in ("x", "dy", "gain", "beta", "w1", "w2", "b1", "b2"):
                t[k].copy_(new[k])
            for k in OUTS:
                t[k].fill_(3.0)
            g.replay()
            torch.cuda.synchronize()
            _block(nsm, h, new, "gelu", "in_out")
            torch.cuda.synchronize()
            for k in OUTS:
                assert torch.equal(t[k], new[k]), (rep, i, k)


def test_capture_needs_a_resident_workspace(nsm):
    import torch
    h = nsm.muon_init(0)
    try:
        t = _block_tensors(100, 128, 264, "in_out", 8)
        g = torch.cuda.CUDAGraph()
        with pytest.raises(nsm.MuonError) as ei:
            with torch.cuda.graph(g):
                nsm.muon_linear_grad_weight(h, t["x"], t["dz"], t["dw1"])
                nsm.muon_layernorm_backward(h, t["dxn"], t["x"], t["gain"], t["mean"], t["rstd"], t["dx"], t["dgain"])
        assert ei.value.status == nsm.MUON_ERR_INVALID_ARG and "capture" in str(ei.value)
        torch.cuda.synchronize()
        assert nsm.muon_workspace_bytes(h) == 0
        nsm.muon_layernorm_backward(h, t["dxn"], t["x"], t["gain"], t["mean"], t["rstd"], t["dx"], t["dgain"])
        torch.cuda.synchronize()
        assert nsm.muon_workspace_bytes(h) > 0
    finally:
        nsm.muon_destroy(h)


def test_offsets_past_32_bits(nsm, h):
    """Views whose last rows lie more than 2^32 bytes from their first: a column
    block of a wide buffer."""
    import torch
    rows, ld, c, n = 70001, 32768, 64, 40
    big = torch.zeros(rows, ld, device="cuda", dtype=torch.bfloat16)
    x = big[:, ld - c:]
    x.normal_()
    xv = x.float()
    pick = [0, 1, 32767, 32768, 65535, 65536, rows - 1]
    g, w = torch.ones(c, device="cuda"), torch.randn(c, n, device="cuda").bfloat16()
    y = big[:, :c]
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    nsm.muon_layernorm_forward(h, x, g, None, y, mean=mean, rstd=rstd)
    ry = torch.nn.functional.layer_norm(xv[pick].double(), (c,))
    assert float((y[pick].double() - ry).abs().max()) <= 2 ** -8 * float(ry.abs().max()) + 1e-4
    o = big[:, c:c + n]
    nsm.muon_linear_forward(h, x, w, o)
    ro = xv[pick].double() @ w.double()
    assert bool(((o[pick].double() - ro).abs() <= 2 ** -8 * ro.abs() + 80 * U * (xv[pick].abs().double() @ w.abs().double())).all())
    dw, db = torch.empty(c, n, device="cuda"), torch.empty(n, device="cuda")
    nsm.muon_linear_grad_weight(h, x, o, dw, db=db)
    rdw = xv.double().t() @ o.double()
    mag = xv.double().abs().t() @ o.double().abs()
    # 70001 rows in float32: each lane's sums run through K / splits additions
    assert bool(((dw.double() - rdw).abs() <= rows * U * mag).all())
    assert bool(((db.double() - o.double().sum(0)).abs() <= rows * U * o.double().abs().sum(0)).all())
    q = nsm.Act8(torch.zeros(rows, ld, dtype=torch.int8, device="cuda")[:, ld - c:],
                 torch.zeros(rows, ld, dtype=torch.uint8, device="cuda")[:, ld - 2:])
    nsm.muon_act_encode(h, x, q)
    back = big[:, 128:128 + c]
    nsm.muon_act_decode(h, q, back)
    rq, re = lo.act8_encode(xv[pick].double().cpu().numpy())
    assert np.array_equal(host(back[pick]), lo.act8_decode(rq, re))
    dw2 = torch.empty_like(dw)
    nsm.muon_linear_grad_weight(h, q, o, dw2)
    r2 = back.double().t() @ o.double()
    assert bool(((dw2.double() - r2).abs() <= rows * U * (back.double().abs().t() @ o.double().abs())).all())
