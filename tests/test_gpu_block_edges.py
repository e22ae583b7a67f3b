"""Calls of the block operators that the definition answers and the other tests do not
make, on the GPU: infinities and NaN beside a mask, a single parameter.  u and h as in
test_gpu_blocks."""

import numpy as np
import pytest

from oracle import block_oracle as bo
from test_gpu_layers import HALF, U, close, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nsm():
    import newton_schulz_matrix_step_amd as m
    return m


@pytest.fixture()
def h(nsm):
    hd = nsm.muon_init(0)
    yield hd
    nsm.muon_destroy(hd)


@pytest.mark.parametrize("p", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("types", [("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("float32", "float32")], ids="-".join)
@pytest.mark.parametrize("cols", [6, 24, 1000, 4095, 9000])
def test_zero_gradient_beside_an_infinite_branch(nsm, h, cols, types, p):
    """e t with e = 0 and an infinite or NaN t is NaN where the element is kept, and
    nothing where it is dropped, with and without a mask drawn."""
    import torch
    torch.manual_seed(4)
    rows, (sst, bst) = 7, (getattr(torch, t) for t in types)
    keep = torch.from_numpy(bo.dropout_factors(rows, cols, p, 9, 10) != 0).cuda()
    ds = torch.randn(rows, cols, device="cuda").to(sst)
    branch = torch.randn(rows, cols, device="cuda").to(bst)
    ds[2, ::3], branch[2, ::3] = 0.0, float("inf")
    ds[4, 1::3], branch[4, 1::3] = -0.0, float("nan")
    gate = torch.ones(cols, device="cuda")
    dx, db, dg = torch.empty_like(ds), torch.empty_like(branch), torch.empty_like(gate)
    nsm.muon_blocknorm_backward(h, dx, ds=ds, branch=branch, dbranch=db, gate=gate, dgate=dg, drop=nsm.Dropout(p, 9, 10))
    want = torch.zeros(cols, dtype=torch.bool, device="cuda")
    want[::3] |= keep[2, ::3]
    want[1::3] |= keep[4, 1::3]
    assert torch.equal(dg.isnan(), want) and not dg.isinf().any()
    assert torch.equal(dx, ds) and bool((db[~keep] == 0).all()) and bool(db.isfinite().all())


@pytest.mark.parametrize("pst", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [7, 1000, 9000])
def test_a_post_bias_alone(nsm, h, cols, pst):
    """A branch's layer norm with a bias and no gain, forward and backward, against the
    float64 oracle.  Bounds: those of the general junction, with every factor 1."""
    rng = np.random.default_rng([11, cols])
    rows, d = 37, 64 + cols / 512
    (x, xv), (o, ov), (ds, dsv) = (dev(rng.normal(size=(rows, cols)), "fp32") for _ in range(3))
    bias, bv = dev(rng.normal(size=cols), pst)
    s, _ = dev(np.zeros((rows, cols)), "fp32")
    mean, rstd = (dev(np.zeros(rows), "fp32")[0] for _ in range(2))
    nsm.muon_blocknorm_forward(h, x, branch=o, s=s, post_norm="layer", post_bias=bias, post_mean=mean, post_rstd=rstd)
    want, wm, wr = bo.junction_stream(xv, ov, "layer", None, bv)
    oh = bo.norm(ov, "layer", 1e-5)[0]
    eo = d * U * (2 * np.abs(oh) + np.abs(ov).mean(1, keepdims=True) * wr[:, None])
    close(host(s), want, eo + 8 * U * (np.abs(oh) + np.abs(bv)) + 2 * U * (np.abs(xv) + np.abs(want)) + U * np.abs(want), "s")
    db, dbias = dev(np.zeros((rows, cols)), "fp32")[0], dev(np.zeros(cols), pst)[0]
    dx = dev(np.zeros((rows, cols)), "fp32")[0]
    nsm.muon_blocknorm_backward(h, dx, ds=ds, branch=o, dbranch=db, post_norm="layer", post_bias=bias, post_mean=mean,
                                post_rstd=rstd, dpost_bias=dbias)
    assert (host(dx) == dsv).all()
    m, r = host(mean), host(rstd)
    g = bo.junction_grad({"post_mean": m, "post_rstd": r}, None, dsv, None, ov, "layer", None, bv)
    close(host(dbias), g["dpost_bias"], (rows + 16) * U * np.abs(dsv).sum(0) + (2 * U + HALF[pst]) * np.abs(g["dpost_bias"]),
          "dpost_bias")
    ah, e = np.abs((ov - m[:, None]) * r[:, None]), np.abs(dsv)
    tol = r[:, None] * ((d + 8) * U * (e.mean(1, keepdims=True) + ah * (e * ah).mean(1, keepdims=True)) + 8 * U * e)
    close(host(db), g["dbranch"], tol + (2 * U + HALF["fp32"]) * np.abs(g["dbranch"]), "dbranch")
