"""The gated products that the GPU tests compare with float64 cover every kernel that the
plan picks for the widths of large models and for sizes of any value."""

import os

import pytest

import block_plan as bp
import block_plan_wide as wide


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    if not os.path.exists(bp.CXX):
        pytest.skip("ROCm clang++ not available")
    return bp.build(tmp_path_factory.mktemp("plan_wide"))


def test_checked_products_cover_every_kernel_of_wide_layers(exe):
    have = set(bp.variants(exe, bp.CASES + wide.CASES))
    assert len(have) == len(set(bp.variants(exe, bp.CASES))) + len(wide.CASES)
    sizes = wide.sweep()
    for c, v in zip(sizes, bp.variants(exe, sizes)):
        assert v in have, (c, v)


def test_ragged_cases_run_the_same_kernels(exe):
    """The GPU test takes a few rows and columns off its cases; these keep their kernels."""
    ragged = [(k, r - 5, i - 8, f - 8, dt, lay) for k, r, i, f, dt, lay in wide.CASES]
    assert bp.variants(exe, ragged) == bp.variants(exe, wide.CASES)
