"""Calls that the binding has to take as the C ABI does, as far as they get without a
GPU: past the checks of shapes and types, up to the device's."""

import pytest
import torch

import newton_schulz_matrix_step_amd as nsm


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", ["post_gain", "post_bias", "gate", "pre_gain", "pre_bias"])
def test_a_junction_may_have_any_one_parameter(name, dt):
    x, p = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=dt)
    r = torch.zeros(4)
    norms = dict(post_norm="layer", pre_norm="layer")
    with pytest.raises(ValueError, match="must all be on one GPU"):
        nsm.muon_blocknorm_forward(0, x, branch=x, s=x, y=x, **norms, **{name: p})
    par = {} if name == "pre_bias" else {name: p}      # (its gradient needs the bias's type alone)
    with pytest.raises(ValueError, match="must all be on one GPU"):
        nsm.muon_blocknorm_backward(0, x, dy=x, s=x, branch=x, dbranch=x, post_mean=r, post_rstd=r, pre_mean=r, pre_rstd=r,
                                    **norms, **par, **{"d" + name: p})


def test_parameters_of_two_types_are_refused():
    x, a, b = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16)
    r = torch.zeros(4)
    with pytest.raises(ValueError, match="pre_gain is|post_bias is"):
        nsm.muon_blocknorm_backward(0, x, dy=x, s=x, branch=x, dbranch=x, post_norm="layer", post_bias=a, post_mean=r,
                                    post_rstd=r, pre_norm="rms", pre_gain=b, pre_rstd=r)
