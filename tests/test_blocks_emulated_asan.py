"""The block operators' kernels and host code under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU, compiled against the layer operators'
stand-in of HIP (tests/emu_layers): every global address a kernel forms is checked
against exactly sized buffers, and the padding between rows against its old value.
Values are not checked here (one thread runs at a time, and the stand-in's matrix
instructions do nothing)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_matrix_step_amd", "csrc")
EMU = os.path.join(ROOT, "tests", "emu_layers")
CXX = "/opt/rocm/lib/llvm/bin/clang++"
SOURCES = ("muon_kernels.hip", "adamw_kernels.hip", "muon_static.hip", "norm_kernels.hip", "linear_kernels.hip",
           "gated_kernels.hip", "blocknorm_kernels.hip", "blocknorm_grad_kernels.hip", "dropout_kernels.hip",
           "muon_api.cpp", "layer_api.cpp", "block_api.cpp")


def _build(tmp_path_factory, name, extra):
    if not os.path.exists(CXX):
        pytest.skip("ROCm clang++ not available")
    out = tmp_path_factory.mktemp(name)
    flags = ["-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
             "-fno-omit-frame-pointer", f"-I{EMU}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
             "-Wno-unused-value", *extra]
    jobs = []
    for src in [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "emu_blocks", "emu_blocks_driver.cpp")]:
        obj = str(out / (os.path.basename(src) + ".o"))
        jobs.append((obj, subprocess.Popen([CXX, *flags, "-x", "c++", src, "-c", "-o", obj])))
    for obj, p in jobs:
        assert p.wait() == 0, obj
    exe = str(out / "emu_blocks_driver")
    subprocess.run([CXX, "-fsanitize=address,undefined", *[o for o, _ in jobs], "-o", exe], check=True)
    return exe


@pytest.fixture(scope="module")
def emu(tmp_path_factory):
    return _build(tmp_path_factory, "emu_blocks", [])


# op, rows, in or cols, hidden, types (0 bf16, 1 float32, 2 float32 stream and bf16 blocks), flags (1 out x in,
# 2 8-bit, 4 no optional arguments, 8 layer norms, 16 no branch, 32 in place), pad, shift
GATED = [("gated", r, i, f, dt, fl, pad, sh)
         for r, i, f in ((1, 8, 8), (1, 1, 1), (1, 512, 264), (5, 72, 136), (130, 200, 128), (129, 131, 67),
                         (64, 128, 640), (300, 96, 40))
         for dt, fl, pad, sh in ((0, 0, 0, 0), (0, 1, 0, 0), (0, 2, 8, 0), (0, 3, 0, 0), (0, 39, 3, 1), (1, 32, 4, 0),
                                 (1, 3, 0, 0), (1, 4, 1, 1))]
NORM = [("norm", r, c, 0, dt, fl, pad, sh)
        for r, c in ((1, 1), (3, 40), (37, 512), (9, 520), (5, 1024), (5, 1500), (6, 2048), (3, 2999), (3, 4096),
                     (2, 8191), (2, 9000))
        for dt, fl, pad, sh in ((0, 0, 0, 0), (0, 10, 8, 0), (0, 44, 3, 1), (1, 42, 0, 0), (1, 20, 1, 1), (2, 8, 0, 0),
                                (2, 2, 1, 1), (2, 26, 4, 0))]
DROP = [("drop", r, c, 0, dt, fl, pad, sh)
        for r, c in ((1, 1), (3, 31), (5, 32), (7, 33), (130, 64), (2, 8200), (1100, 3))
        for dt, fl, pad, sh in ((0, 0, 0, 0), (1, 4, 0, 0), (0, 36, 8, 0), (1, 32, 3, 1), (0, 0, 1, 1))]


def _run(exe, case, verbose=False):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    if verbose:
        env["EMU_VERBOSE"] = "1"
    r = subprocess.run([exe, *[str(v) for v in case]], capture_output=True, text=True, env=env, timeout=900)
    assert "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
    assert "runtime error" not in r.stderr, r.stderr[-3000:]
    assert r.returncode == 0, (r.stdout, r.stderr[-2000:])
    return r


def _all(exe, cases):
    seen = ""
    for case in cases:
        try:
            seen += _run(exe, case, verbose=True).stderr
        except AssertionError as e:
            raise AssertionError(f"{case}: {e}") from e
    return seen


@pytest.mark.parametrize("cases,kernels", [
    (GATED, ("linear_tile_kernel", "gated_join_kernel", "linear_pack_kernel")),
    (NORM, ("blocknorm_kernel", "blocknorm_grad_kernel", "blocknorm_long_kernel", "blocknorm_grad_long_kernel",
            "blocknorm_join_kernel")),
    (DROP, ("dropout_kernel",)),
], ids=["gated", "norm", "drop"])
def test_block_kernels_stay_in_bounds(emu, cases, kernels):
    seen = _all(emu, cases)
    for k in kernels:
        assert k in seen, k


# The 128- and 256-wide kernels, which the library gives only to larger products.
EDGE_CASES = [("gated", r, i, f, dt, fl, pad, sh)
              for r, i, f in ((1, 8, 8), (130, 200, 264), (257, 136, 300), (300, 1000, 520))
              for dt, fl, pad, sh in ((0, 0, 0, 0), (0, 1, 8, 0), (0, 2, 0, 0), (0, 3, 0, 0), (0, 7, 3, 1), (1, 3, 0, 0))]


@pytest.mark.parametrize("edge,kernel", [(128, "linear_tile_kernel"), (256, "linear_pp_kernel")])
def test_wider_tiles_stay_in_bounds(tmp_path_factory, edge, kernel):
    exe = _build(tmp_path_factory, f"emu_blocks_{edge}", [f"-DMUON_LINEAR_EDGE={edge}"])
    assert kernel in _all(exe, EDGE_CASES)


def test_refusals_enqueue_nothing(emu):
    """Null and misaligned pointers, sizes, leading dimensions, dtypes, aliasing,
    flags, scales, probabilities and failing allocations: the status each call must
    return, an error text, and no launch."""
    r = _run(emu, ("refuse",))
    assert "refusals wrong 0" in r.stdout, r.stdout
