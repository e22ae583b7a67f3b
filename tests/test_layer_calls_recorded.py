"""Host side of the layer operators on calls whose launches are written down
instead of run: what is refused, what is launched and what workspace is held."""

import os

import pytest

import layer_record as rec

OK, INVALID, OOM = 0, 1, 4


@pytest.fixture(scope="module")
def call(tmp_path_factory):
    if not os.path.exists(rec.CXX):
        pytest.skip("ROCm clang++ not available")
    exe = rec.build(tmp_path_factory.mktemp("record"))
    return lambda *lines: rec.calls(exe, lines)


@pytest.mark.parametrize("line", ["ln 0 40 0 null bias y8", "fwd 0 40 72 null bias res act=1 z8", "fwd 0 40 72 null act=2 z",
                                  "dx 0 40 72 null act=1 z8 actout", "dx 0 40 72 null act=2 z actout add", "dx 0 40 72 null",
                                  "enc 0 40 0 null", "dec 0 40 0 null"])
def test_no_rows_is_no_call(call, line):
    """A batch without rows is taken, with the null addresses of empty tensors,
    whatever the optional arguments, and enqueues nothing."""
    r, = call(line)
    assert r["status"] == OK and r["launches"] == [], r


@pytest.mark.parametrize("line", ["dw 0 40 72 null db", "dw 0 40 72 null x8 db acc", "lngrad 0 40 0 null add"])
def test_no_rows_still_writes_parameter_gradients(call, line):
    r, = call(line)
    assert r["status"] == OK and len(r["launches"]) == 1, r


@pytest.mark.parametrize("line", ["dx 4 40 72 act=1", "dx 4 40 72 actout", "dx 0 40 72 act=7", "dx 0 40 72 act=1 null pad=-1"])
def test_missing_pre_activation_is_refused(call, line):
    r, = call(line)
    assert r["status"] == INVALID and r["launches"] == [], r


@pytest.mark.gpu
def test_empty_tensors_with_an_activation():
    import torch

    import newton_schulz_matrix_step_amd as nsm
    h = nsm.muon_init(0)
    try:
        def e(n):
            return torch.empty(0, n, device="cuda", dtype=torch.bfloat16)

        w = torch.ones(40, 72, device="cuda", dtype=torch.bfloat16)
        for z in (e(40), nsm.Act8.empty(0, 40)):
            nsm.muon_linear_grad_input(h, e(72), w, e(40), act="gelu", z=z, act_out=e(40), add=e(40))
        nsm.muon_linear_forward(h, e(40), w, e(72), act="gelu", z_out=nsm.Act8.empty(0, 72))
        nsm.muon_act_encode(h, e(40), nsm.Act8.empty(0, 40))
        nsm.muon_act_decode(h, nsm.Act8.empty(0, 40), e(40))
        torch.cuda.synchronize()
    finally:
        nsm.muon_destroy(h)
