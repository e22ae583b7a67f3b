"""The list of products that the GPU tests compare with float64 covers every
kernel that the plan picks over a wide range of sizes: a refit of the plan's time
model that leaves a kernel without a checked product fails here."""

import os

import pytest

import layer_plan_cases as cases
import layer_record as rec


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    if not os.path.exists(rec.CXX):
        pytest.skip("ROCm clang++ not available")
    return rec.build(tmp_path_factory.mktemp("record"))


def test_checked_products_cover_every_kernel(exe):
    have = {cases.variant(line, r) for line, r in zip(cases.CASES, rec.calls(exe, cases.CASES))}
    assert len(have) == len(cases.CASES)
    lines = cases.sweep()
    for i in range(0, len(lines), 20000):
        part = lines[i:i + 20000]
        for line, r in zip(part, rec.calls(exe, part)):
            assert r["status"] == 0, (line, r)
            assert cases.variant(line, r) in have, (line, cases.variant(line, r))


def test_streamed_activations_are_covered(exe):
    """act(z) of input gradients past the size from which it is streamed, and under
    it, on the 256-wide tiles and on narrower ones."""
    seen = set()
    for line in cases.CASES + cases.STREAMS:
        if line.startswith("dx"):
            k = cases.product(rec.calls(exe, [line + " z act=1 actout"])[0])
            if k["splits"] == 1:
                seen.add((k["tile"] == 256, bool(k["act_stream"])))
    assert seen == {(False, False), (False, True), (True, False), (True, True)}
