"""The gated products of wide layers (block_plan_wide.CASES) against float64 products on
the GPU: the checks and bounds of test_gpu_block_kernels."""

import pytest

import block_plan_wide as wide
import test_gpu_block_kernels as base
from test_gpu_block_kernels import h, nsm  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", wide.CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_wide_product(nsm, h, case, ragged):  # noqa: F811
    base.test_product(nsm, h, case, ragged)
