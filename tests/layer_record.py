"""Builds the launch-recording host build of the library (tests/emu_record) and
makes layer calls in it: any sizes, nothing read or run."""

import json
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_matrix_step_amd", "csrc")
EMU = os.path.join(ROOT, "tests", "emu_record")
CXX = "/opt/rocm/lib/llvm/bin/clang++"
SOURCES = ("muon_kernels.hip", "adamw_kernels.hip", "muon_static.hip", "norm_kernels.hip", "linear_kernels.hip",
           "muon_api.cpp", "layer_api.cpp")


def build(out_dir) -> str:
    """The driver's path."""
    flags = ["-O1", "-std=c++17", f"-I{EMU}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-Wno-unused-value"]
    jobs = []
    for src in [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(EMU, "record_driver.cpp")]:
        obj = os.path.join(str(out_dir), os.path.basename(src) + ".o")
        jobs.append((obj, subprocess.Popen([CXX, *flags, "-x", "c++", src, "-c", "-o", obj])))
    for obj, p in jobs:
        assert p.wait() == 0, obj
    exe = os.path.join(str(out_dir), "record_driver")
    subprocess.run([CXX, *[o for o, _ in jobs], "-o", exe], check=True)
    return exe


def calls(exe, lines):
    """One dict (status, error, workspace, launches) for each call among `lines`."""
    r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return [json.loads(v) for v in r.stdout.splitlines()]
