"""Passes over very many rows go in several launches: the same code with slices
of 512 threads, on sizes that fit a test."""

import pytest

import test_layers_emulated_asan as emulated


def test_slices_stay_in_bounds(tmp_path_factory):
    exe = emulated._build(tmp_path_factory, "emu_layers_slices", ["-DMUON_SLICE_THREADS=512"])
    whole = emulated._build(tmp_path_factory, "emu_layers_whole", [])
    more = 0
    for case in (("act", 900, 64, 0, 0, 0, 0, 0), ("act", 700, 33, 0, 1, 0, 3, 1), ("act", 5, 8200, 0, 0, 0, 8, 0),
                 ("lin", 130, 200, 131, 0, 7, 3, 1), ("lin", 300, 96, 40, 1, 3, 0, 0), ("lin", 129, 131, 67, 0, 2, 0, 0)):
        a, b = (emulated._run(e, case, verbose=True).stderr.count("launch") for e in (exe, whole))
        assert a >= b
        more += a > b
    assert more >= 3


@pytest.mark.gpu
def test_product_of_more_than_2_30_rows():
    """2^30 rows and some of a narrow product: as many 64-wide tiles as no launch
    can have.  Checked at rows around each boundary of the addressing, against
    float64 (a sum of 8 products in float32, then one rounding)."""
    import torch

    import newton_schulz_matrix_step_amd as nsm
    rows, k, n = (1 << 30) + 77, 8, 8
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    h = nsm.muon_init(0)
    try:
        x = torch.empty(rows, k, device="cuda", dtype=torch.bfloat16).uniform_(-1, 1)
        w = torch.randn(k, n, device="cuda").bfloat16()
        y = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16)
        y[-200:] = 7.0
        nsm.muon_linear_forward(h, x, w, y)
        pick = torch.cat([torch.arange(max(0, c - 70), min(rows, c + 70)) for c in
                          (0, 1 << 24, 1 << 27, 1 << 28, 1 << 29, 3 << 28, 1 << 30, rows)]).cuda()
        xd = x[pick].double()
        want, mag = xd @ w.double(), xd.abs() @ w.double().abs()
        got = y[pick].double()
        assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 24 * 2.0 ** -24 * mag).all())
    finally:
        nsm.muon_destroy(h)
        del x, y
        torch.cuda.empty_cache()
