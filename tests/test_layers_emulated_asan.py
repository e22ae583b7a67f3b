"""The layer operators' kernels and host code under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU, compiled against a stand-in of HIP
(tests/emu_layers): every global address a kernel forms is checked against
exactly sized buffers, and the padding between rows against its old value.
Values are not checked here (the stand-in's matrix instructions do nothing)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_matrix_step_amd", "csrc")
EMU = os.path.join(ROOT, "tests", "emu_layers")
CXX = "/opt/rocm/lib/llvm/bin/clang++"


def _build(tmp_path_factory, name, extra):
    if not os.path.exists(CXX):
        pytest.skip("ROCm clang++ not available")
    out = tmp_path_factory.mktemp(name)
    flags = ["-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
             "-fno-omit-frame-pointer", f"-I{EMU}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
             "-Wno-unused-value", *extra]
    jobs = []
    for src in ("muon_kernels.hip", "adamw_kernels.hip", "muon_static.hip", "norm_kernels.hip", "linear_kernels.hip",
                "muon_api.cpp", "layer_api.cpp"):
        obj = str(out / (src + ".o"))
        jobs.append((obj, subprocess.Popen([CXX, *flags, "-x", "c++", os.path.join(CSRC, src), "-c", "-o", obj])))
    obj = str(out / "driver.o")
    jobs.append((obj, subprocess.Popen([CXX, *flags, os.path.join(EMU, "emu_layers_driver.cpp"), "-c", "-o", obj])))
    for obj, p in jobs:
        assert p.wait() == 0, obj
    exe = str(out / "emu_layers_driver")
    subprocess.run([CXX, "-fsanitize=address,undefined", *[o for o, _ in jobs], "-o", exe], check=True)
    return exe


@pytest.fixture(scope="module")
def emu(tmp_path_factory):
    return _build(tmp_path_factory, "emu_layers", [])


# op, rows, cols / in, out, dtype (0 bf16, 1 f32), flags (1 out x in, 2 8-bit, 4 no optional arguments), pad, shift
CASES = [("ln", r, c, 0, dt, fl, pad, sh)
         for r, c in ((1, 1), (3, 40), (37, 512), (9, 520), (5, 1024), (5, 1500), (6, 2048), (3, 3000), (3, 4096),
                      (2, 8192), (2, 9000), (2, 16384), (2, 17000))
         for dt, fl, pad, sh in ((0, 0, 0, 0), (1, 2, 0, 0), (0, 2, 8, 0), (0, 6, 3, 1))]
CASES += [("lin", r, i, o, dt, fl, pad, sh)
          for r, i, o in ((1, 8, 8), (1, 1, 1), (1, 512, 264), (5, 72, 136), (130, 200, 128), (129, 131, 67),
                          (64, 128, 640), (300, 96, 40))
          for dt, fl, pad, sh in ((0, 0, 0, 0), (0, 1, 0, 0), (0, 2, 8, 0), (0, 3, 0, 0), (0, 7, 3, 1), (1, 0, 4, 0),
                                  (1, 3, 0, 0), (1, 4, 1, 1))]
CASES += [("act", r, c, 0, dt, 0, pad, sh)
          for r, c in ((1, 1), (3, 31), (5, 32), (7, 33), (2, 1000), (130, 64), (2, 8200))
          for dt, pad, sh in ((0, 0, 0), (1, 0, 0), (0, 8, 0), (1, 3, 1))]


def _run(exe, case, verbose=False):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0")
    if verbose:
        env["EMU_VERBOSE"] = "1"
    r = subprocess.run([exe, *[str(v) for v in case]], capture_output=True, text=True, env=env, timeout=900)
    assert "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
    assert "runtime error" not in r.stderr, r.stderr[-3000:]
    assert r.returncode == 0, (r.stdout, r.stderr[-2000:])
    return r


@pytest.mark.parametrize("op", ["ln", "lin", "act"])
def test_layer_kernels_stay_in_bounds(emu, op):
    for case in CASES:
        if case[0] == op:
            try:
                _run(emu, case)
            except AssertionError as e:
                raise AssertionError(f"{case}: {e}") from e


# The 128- and 256-wide kernels, which the library gives only to larger products.
EDGE_CASES = [("lin", r, i, o, dt, fl, pad, sh)
              for r, i, o in ((1, 8, 8), (130, 200, 264), (257, 136, 300), (300, 1000, 520))
              for dt, fl, pad, sh in ((0, 0, 0, 0), (0, 1, 8, 0), (0, 2, 0, 0), (0, 3, 0, 0), (0, 7, 3, 1), (1, 3, 0, 0))]


@pytest.mark.parametrize("edge,kernel", [(128, "linear_tile_kernel"), (256, "linear_pp_kernel")])
def test_wider_tiles_stay_in_bounds(tmp_path_factory, edge, kernel):
    exe = _build(tmp_path_factory, f"emu_layers_{edge}", [f"-DMUON_LINEAR_EDGE={edge}"])
    seen = ""
    for case in EDGE_CASES:
        try:
            seen += _run(exe, case, verbose=True).stderr
        except AssertionError as e:
            raise AssertionError(f"{case}: {e}") from e
    assert kernel in seen


def test_refusals_enqueue_nothing(emu):
    """Null and misaligned pointers, sizes, leading dimensions, dtypes, aliasing,
    flags and failing allocations: the status each call must return, an error
    text, and no launch."""
    r = _run(emu, ("refuse",))
    assert "refusals wrong 0" in r.stdout, r.stdout
