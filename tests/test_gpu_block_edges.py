"""Calls of the block operators that the definition answers and the other tests do not
make, on the GPU: infinities and NaN beside a mask."""

import pytest

from oracle import block_oracle as bo

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
