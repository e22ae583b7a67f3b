"""Every kernel that the plan of the gated products picks, against float64 products on
the GPU.  Sizes are those of block_plan.CASES less a few rows and columns where that
keeps the plan, so that tiles end ragged."""

import pytest

import block_plan as bp

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


def silu(z):
    import torch
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s))


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", bp.CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_product(nsm, h, case, ragged):
    """Bounds as in test_gpu_blocks: a sum of n products within (n + 8) u of their
    magnitudes, through a factor's error where there is one, and one rounding."""
    import torch
    kind, rows, i, f, dt, oi = case
    if ragged:                       # 8-element runs cut at the tiles' ends
        rows, i, f = max(1, rows - 5), i - 8 if i > 64 else i, f - 8
    torch.manual_seed(rows + i + f)
    t = torch.float32 if dt else torch.bfloat16
    half = U if dt else 2.0 ** -8
    lay = "out_in" if oi else "in_out"

    def rnd(*s, std=1.0):
        return (torch.randn(*s, device="cuda") * std).to(t)

    def weight(a, b):
        return rnd(b, a, std=a ** -0.5) if oi else rnd(a, b, std=a ** -0.5)

    def io(w):
        return w.double().t().contiguous() if oi else w.double()

    def check(got, want, tol, what):
        bad = (got.double() - want).abs() - tol - (2 * U + half) * want.abs()
        assert float(bad.max()) <= 0, (what, float(bad.max()))

    def product(a, b):
        return a @ b, (a.shape[1] + 8) * U * (a.abs() @ b.abs())

    if kind == "fwd":
        x, wg, wu = rnd(rows, i), weight(i, f), weight(i, f)
        y, zo = torch.empty(rows, f, device="cuda", dtype=t), [torch.empty(rows, f, device="cuda", dtype=t) for _ in range(2)]
        nsm.muon_gated_forward(h, x, wg, wu, y, gate_out=zo[0], up_out=zo[1], w_layout=lay)
        (zg, tg), (zu, tu) = product(x.double(), io(wg)), product(x.double(), io(wu))
        a = silu(zg)[0]
        ta = 1.13 * tg + 8 * U * (1 + a.abs())
        check(zo[0], zg, tg, "gate")
        check(zo[1], zu, tu, "up")
        check(y, a * zu, ta * zu.abs() + (a.abs() + ta) * tu, "h")
    elif kind == "dh":
        dy, wd, zg, zu = rnd(rows, i), weight(f, i), rnd(rows, f), rnd(rows, f)
        dg, du, ho = (torch.empty(rows, f, device="cuda", dtype=t) for _ in range(3))
        nsm.muon_gated_grad_hidden(h, dy, wd, zg, zu, dg, du, h_out=ho, w_layout=lay)
        dh, td = product(dy.double(), io(wd).t().contiguous())
        a, d = silu(zg.double())
        u, ta = zu.double(), 8 * U * (1 + a.abs())
        check(dg, dh * u * d, u.abs() * (td * (d.abs() + 16 * U) + dh.abs() * 16 * U) + U * (dh * u * d).abs(), "dgate")
        check(du, dh * a, td * (a.abs() + ta) + dh.abs() * ta, "dup")
        check(ho, a * u, ta * u.abs(), "h")
    elif kind == "dx":
        dg, du, wg, wu = rnd(rows, f), rnd(rows, f), weight(i, f), weight(i, f)
        dx = torch.empty(rows, i, device="cuda", dtype=t)
        nsm.muon_gated_grad_input(h, dg, du, wg, wu, dx, w_layout=lay)
        want, tol = product(torch.cat([dg, du], 1).double(), torch.cat([io(wg), io(wu)], 1).t().contiguous())
        check(dx, want, tol, "dx")
    else:
        x, dg, du = rnd(rows, i), rnd(rows, f), rnd(rows, f)
        dw = [torch.empty(*((f, i) if oi else (i, f)), device="cuda", dtype=t) for _ in range(2)]
        db = [torch.empty(f, device="cuda") for _ in range(2)]
        nsm.muon_gated_grad_weight(h, x, dg, du, *dw, db_gate=db[0], db_up=db[1], w_layout=lay)
        for w, b, dz, nm in ((dw[0], db[0], dg, "gate"), (dw[1], db[1], du, "up")):
            want, tol = product(x.double().t().contiguous(), dz.double())
            check(w.t() if oi else w, want, tol, "dw " + nm)
            s = dz.double().sum(0)
            assert float(((b.double() - s).abs() - (rows + 8) * U * dz.double().abs().sum(0) - 2 * U * s.abs()).max()) <= 0
