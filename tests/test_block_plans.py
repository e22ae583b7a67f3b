"""The list of gated products that the GPU tests compare with float64 covers every
kernel that the plan picks over a wide range of sizes: a refit of the plan's time model
that leaves a kernel without a checked product fails here."""

import os

import pytest

import block_plan as bp


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    if not os.path.exists(bp.CXX):
        pytest.skip("ROCm clang++ not available")
    return bp.build(tmp_path_factory.mktemp("plan"))


def test_checked_products_cover_every_kernel(exe):
    have = set(bp.variants(exe, bp.CASES))
    sweep = bp.sweep()
    for c, v in zip(sweep, bp.variants(exe, sweep)):
        assert v in have, (c, v)


def test_splits_leave_no_part_empty(exe):
    """Every split has k blocks of its own, and no more splits than two workgroups a CU
    ask for."""
    import subprocess
    sweep = [c for c in bp.sweep() if c[5] == 0]
    r = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in sweep) + "\n", capture_output=True, text=True,
                       check=True)
    for (kind, rows, i, f, dt, _), line in zip(sweep, r.stdout.splitlines()):
        tile, deep, s = (int(v) for v in line.split())
        bk = 32 if dt else 64
        m, n, k, mult = {"fwd": (rows, 2 * f, i, 1), "dh": (rows, f, i, 1), "dx": (rows, i, f, 2), "dw": (i, 2 * f, rows, 1)}[kind]
        nkb = -(-k // bk) * mult
        per = -(-nkb // s)
        assert (s - 1) * per < nkb and s <= 64, (kind, rows, i, f, dt)
        assert not deep or -(-m // tile) * -(-n // tile) * s <= 256 + -(-m // tile) * s
