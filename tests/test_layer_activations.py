"""The activations of the linear products' epilogues at infinite and NaN
pre-activations: forward and backward agree, on the limits of the definition
(GELU: value 0 and derivative 0 at -infinity, infinity and 1 at +infinity;
squared ReLU: 0 and 0, infinity and infinity), and a NaN stays one."""

import math
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_matrix_step_amd", "csrc")
EMU = os.path.join(ROOT, "tests", "emu_layers")
CXX = "/opt/rocm/lib/llvm/bin/clang++"
INF = math.inf
LIMITS = {"gelu": {INF: (INF, 1.0), -INF: (0.0, 0.0)}, "relu_sq": {INF: (INF, INF), -INF: (0.0, 0.0)}}
CODES = {"gelu": 1, "relu_sq": 2}


@pytest.fixture(scope="module")
def host_acts(tmp_path_factory):
    """f(act, zs): forward values, backward values and derivatives of the device code built for the host."""
    if not os.path.exists(CXX):
        pytest.skip("ROCm clang++ not available")
    exe = str(tmp_path_factory.mktemp("acts") / "activations")
    subprocess.run([CXX, "-O1", "-std=c++17", f"-I{EMU}", f"-I{CSRC}", "-Wno-unused-value",
                    os.path.join(EMU, "activations.cpp"), "-o", exe], check=True)

    def run(act, zs):
        text = "".join(f"{CODES[act]} {float(z)!r}\n" for z in zs)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        return np.array([line.split() for line in r.stdout.splitlines()]).astype(np.float32).T

    return run


@pytest.mark.parametrize("act", ["gelu", "relu_sq"])
def test_limits_and_nan(host_acts, act):
    for z, (v, d) in LIMITS[act].items():
        got = host_acts(act, [z])[:, 0]
        assert got[0] == v and got[1] == v and got[2] == d, (z, got)
    assert np.isnan(host_acts(act, [math.nan])).all()


def test_forward_and_backward_values_agree(host_acts):
    """The clamps move no finite value: both sides against float64, within the
    few float32 units of their arithmetic, and beyond |z| = 30 exactly the limit."""
    zs = np.concatenate([np.linspace(-30, 30, 6001), [-9.0, 9.0, -14.0, -1e3, 1e3, -3e38, 3e38]]).astype(np.float32)
    fwd, bwd, der = host_acts("gelu", zs)
    z = zs.astype(np.float64)
    k = math.sqrt(2 / math.pi)
    t = np.tanh(k * (z + 0.044715 * z ** 3))
    want = 0.5 * z * (1 + t)
    dwant = 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    tol = 8 * 2.0 ** -24
    fwd, bwd, der = (t.astype(np.float64) for t in (fwd, bwd, der))
    assert np.all(np.abs(fwd - want) <= tol * (1 + np.abs(want)))
    assert np.all(np.abs(bwd - want) <= tol * (1 + np.abs(want)))
    big = np.abs(z) > 30
    assert np.all(np.abs(der - dwant)[~big] <= 16 * 2.0 ** -24 * 2)
    assert np.array_equal(fwd[big], np.where(z[big] > 0, z[big], 0)) and np.array_equal(bwd[big], fwd[big])
    assert np.array_equal(der[big], (z[big] > 0).astype(float))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "relu_sq"])
@pytest.mark.parametrize("st", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,n", [(20, 13), (40, 64), (300, 264), (4096, 4096)])
def test_epilogues_at_infinities(act, st, rows, n):
    """Through the products: z = 0 W + bias with infinite biases forward, z itself
    infinite backward; the epilogues by element, in vectors and (4096) of the
    widest tiles."""
    import torch

    import newton_schulz_matrix_step_amd as nsm
    dt = torch.bfloat16 if st == "bf16" else torch.float32
    h = nsm.muon_init(0)
    try:
        row = torch.tensor([1.0, INF, -INF, -2.0, math.nan], device="cuda").repeat(n // 5 + 1)[:n].to(dt)
        x, w = torch.zeros(rows, 64, device="cuda", dtype=dt), torch.ones(64, n, device="cuda", dtype=dt)
        y = torch.empty(rows, n, device="cuda", dtype=dt)
        nsm.muon_linear_forward(h, x, w, y, bias=row, act=act)
        z = row.expand(rows, n).contiguous()
        dy, wt = torch.zeros(rows, 64, device="cuda", dtype=dt), torch.ones(n, 64, device="cuda", dtype=dt)
        dy[:, 0] = 1.0
        dx, v = torch.empty_like(y), torch.empty_like(y)
        nsm.muon_linear_grad_input(h, dy, wt, dx, act=act, z=z, act_out=v)
        for s, (want, der) in LIMITS[act].items():
            at = row == s
            for got, what, r in ((y, "y", want), (v, "act_out", want), (dx, "dx", der)):
                assert bool((got[:, at] == r).all()), (what, s, got[0, at][0])
        nan = torch.isnan(row)
        for got in (y, v, dx):
            assert bool(torch.isnan(got[:, nan]).all())
            assert not bool(torch.isnan(got[:, ~nan]).any())
        assert bool(((y - v)[:, row.abs() < 10].float().abs() < 2.0 ** -7).all())
    finally:
        nsm.muon_destroy(h)
