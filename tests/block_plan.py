"""The gated products that the GPU tests compare with float64, one for every kernel
that the plan picks (tile edge, LDS depth, split or not, for each product, layout and
type), and the plan itself in a host build."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "newton_schulz_matrix_step_amd", "csrc")
CXX = "/opt/rocm/lib/llvm/bin/clang++"
SOURCES = ("muon_kernels.hip", "adamw_kernels.hip", "muon_static.hip", "norm_kernels.hip", "linear_kernels.hip",
           "gated_kernels.hip", "muon_api.cpp", "layer_api.cpp")


def build(out_dir) -> str:
    flags = ["-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'tests', 'emu_layers')}", f"-I{os.path.join(ROOT, 'include')}",
             f"-I{CSRC}", "-Wno-unused-value"]
    jobs = []
    for src in [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "tests", "emu_blocks", "plan_driver.cpp")]:
        obj = os.path.join(str(out_dir), os.path.basename(src) + ".o")
        jobs.append((obj, subprocess.Popen([CXX, *flags, "-x", "c++", src, "-c", "-o", obj])))
    for obj, p in jobs:
        assert p.wait() == 0, obj
    exe = os.path.join(str(out_dir), "plan_driver")
    subprocess.run([CXX, *[o for o, _ in jobs], "-o", exe], check=True)
    return exe


def variants(exe, cases):
    """(product, type, layout, tile, depth, split or not) of each case."""
    text = "\n".join(" ".join(str(v) for v in c) for c in cases) + "\n"
    r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=600, check=True)
    out = []
    for c, line in zip(cases, r.stdout.splitlines()):
        tile, deep, splits = (int(v) for v in line.split())
        out.append((c[0], c[4], c[5], tile, deep, splits > 1))
    assert len(out) == len(cases)
    return out


def sweep():
    """Sizes from one row to large products."""
    rows = (1, 16, 100, 300, 700, 1024, 1500, 2048, 4096, 6000, 8192, 16384)
    return [(k, r, i, f, dt, lay) for k in ("fwd", "dh", "dx", "dw") for r in rows
            for i in (64, 256, 512, 768, 1024, 2048, 4096) for f in (64, 352, 704, 1408, 2048, 2816, 5632, 11264)
            for dt in (0, 1) for lay in (0, 1)]


# product, rows, in (dh: out), hidden, type, layout
CASES = [
    ('dh', 1500, 64, 704, 0, 0),
    ('dh', 1, 2048, 2816, 0, 0),
    ('dh', 1, 64, 64, 0, 0),
    ('dh', 1, 2048, 64, 0, 0),
    ('dh', 4096, 64, 2048, 0, 0),
    ('dh', 1024, 64, 2816, 0, 0),
    ('dh', 16384, 64, 2048, 0, 0),
    ('dh', 8192, 64, 2048, 0, 0),
    ('dh', 1500, 64, 704, 0, 1),
    ('dh', 1, 2048, 2816, 0, 1),
    ('dh', 1, 64, 64, 0, 1),
    ('dh', 1, 2048, 64, 0, 1),
    ('dh', 4096, 64, 2048, 0, 1),
    ('dh', 1024, 64, 2816, 0, 1),
    ('dh', 16384, 64, 2048, 0, 1),
    ('dh', 8192, 64, 2048, 0, 1),
    ('dh', 1500, 64, 704, 1, 0),
    ('dh', 1, 1024, 5632, 1, 0),
    ('dh', 1, 64, 64, 1, 0),
    ('dh', 1, 512, 64, 1, 0),
    ('dh', 300, 64, 11264, 1, 0),
    ('dh', 100, 1024, 11264, 1, 0),
    ('dh', 1500, 64, 1408, 1, 0),
    ('dh', 100, 1024, 2816, 1, 0),
    ('dh', 1500, 64, 704, 1, 1),
    ('dh', 1, 1024, 5632, 1, 1),
    ('dh', 1, 64, 64, 1, 1),
    ('dh', 1, 512, 64, 1, 1),
    ('dh', 300, 64, 11264, 1, 1),
    ('dh', 100, 1024, 11264, 1, 1),
    ('dh', 1500, 64, 1408, 1, 1),
    ('dh', 100, 1024, 2816, 1, 1),
    ('dw', 1, 768, 704, 0, 0),
    ('dw', 4096, 64, 352, 0, 0),
    ('dw', 1, 64, 64, 0, 0),
    ('dw', 1500, 64, 64, 0, 0),
    ('dw', 1, 768, 2816, 0, 0),
    ('dw', 6000, 256, 2816, 0, 0),
    ('dw', 1, 64, 11264, 0, 0),
    ('dw', 4096, 512, 352, 0, 0),
    ('dw', 2048, 2048, 11264, 0, 0),
    ('dw', 16384, 4096, 704, 0, 0),
    ('dw', 700, 4096, 2048, 0, 0),
    ('dw', 8192, 1024, 2048, 0, 0),
    ('dw', 1, 768, 704, 0, 1),
    ('dw', 4096, 64, 352, 0, 1),
    ('dw', 1, 64, 64, 0, 1),
    ('dw', 1500, 64, 64, 0, 1),
    ('dw', 1, 768, 2816, 0, 1),
    ('dw', 6000, 256, 2816, 0, 1),
    ('dw', 1, 64, 11264, 0, 1),
    ('dw', 4096, 512, 352, 0, 1),
    ('dw', 2048, 2048, 11264, 0, 1),
    ('dw', 16384, 4096, 704, 0, 1),
    ('dw', 700, 4096, 2048, 0, 1),
    ('dw', 8192, 1024, 2048, 0, 1),
    ('dw', 1, 768, 704, 1, 0),
    ('dw', 1500, 64, 2816, 1, 0),
    ('dw', 1, 64, 64, 1, 0),
    ('dw', 700, 64, 64, 1, 0),
    ('dw', 1, 768, 2816, 1, 0),
    ('dw', 1024, 256, 2816, 1, 0),
    ('dw', 1, 768, 1408, 1, 0),
    ('dw', 1500, 256, 704, 1, 0),
    ('dw', 1, 768, 704, 1, 1),
    ('dw', 1500, 64, 2816, 1, 1),
    ('dw', 1, 64, 64, 1, 1),
    ('dw', 700, 64, 64, 1, 1),
    ('dw', 1, 768, 2816, 1, 1),
    ('dw', 1024, 256, 2816, 1, 1),
    ('dw', 1, 768, 1408, 1, 1),
    ('dw', 1500, 256, 704, 1, 1),
    ('dx', 6000, 768, 64, 0, 0),
    ('dx', 1, 768, 5632, 0, 0),
    ('dx', 1, 64, 352, 0, 0),
    ('dx', 1, 64, 5632, 0, 0),
    ('dx', 1500, 4096, 64, 0, 0),
    ('dx', 300, 1024, 11264, 0, 0),
    ('dx', 1, 64, 64, 0, 0),
    ('dx', 1, 64, 704, 0, 0),
    ('dx', 8192, 4096, 704, 0, 0),
    ('dx', 4096, 4096, 352, 0, 0),
    ('dx', 700, 2048, 11264, 0, 0),
    ('dx', 6000, 768, 64, 0, 1),
    ('dx', 1, 768, 5632, 0, 1),
    ('dx', 1, 64, 352, 0, 1),
    ('dx', 1, 64, 5632, 0, 1),
    ('dx', 1500, 4096, 64, 0, 1),
    ('dx', 300, 1024, 11264, 0, 1),
    ('dx', 1, 64, 64, 0, 1),
    ('dx', 1, 64, 704, 0, 1),
    ('dx', 8192, 4096, 704, 0, 1),
    ('dx', 4096, 4096, 352, 0, 1),
    ('dx', 700, 2048, 11264, 0, 1),
    ('dx', 1500, 768, 64, 1, 0),
    ('dx', 6000, 64, 704, 1, 0),
    ('dx', 1, 64, 64, 1, 0),
    ('dx', 1, 64, 352, 1, 0),
    ('dx', 6000, 768, 64, 1, 0),
    ('dx', 300, 4096, 704, 1, 0),
    ('dx', 700, 4096, 64, 1, 0),
    ('dx', 700, 512, 704, 1, 0),
    ('dx', 1500, 768, 64, 1, 1),
    ('dx', 6000, 64, 704, 1, 1),
    ('dx', 1, 64, 64, 1, 1),
    ('dx', 1, 64, 352, 1, 1),
    ('dx', 6000, 768, 64, 1, 1),
    ('dx', 300, 4096, 704, 1, 1),
    ('dx', 700, 4096, 64, 1, 1),
    ('dx', 700, 512, 704, 1, 1),
    ('fwd', 1, 64, 11264, 0, 0),
    ('fwd', 1, 2048, 1408, 0, 0),
    ('fwd', 1, 64, 64, 0, 0),
    ('fwd', 1, 2048, 64, 0, 0),
    ('fwd', 300, 64, 5632, 0, 0),
    ('fwd', 1500, 4096, 704, 0, 0),
    ('fwd', 700, 64, 1408, 0, 0),
    ('fwd', 8192, 768, 2048, 0, 0),
    ('fwd', 4096, 512, 2048, 0, 0),
    ('fwd', 2048, 4096, 2048, 0, 0),
    ('fwd', 1, 64, 11264, 0, 1),
    ('fwd', 1, 2048, 1408, 0, 1),
    ('fwd', 1, 64, 64, 0, 1),
    ('fwd', 1, 2048, 64, 0, 1),
    ('fwd', 300, 64, 5632, 0, 1),
    ('fwd', 1500, 4096, 704, 0, 1),
    ('fwd', 700, 64, 1408, 0, 1),
    ('fwd', 8192, 768, 2048, 0, 1),
    ('fwd', 4096, 512, 2048, 0, 1),
    ('fwd', 1, 64, 11264, 1, 0),
    ('fwd', 1, 1024, 2816, 1, 0),
    ('fwd', 1, 64, 64, 1, 0),
    ('fwd', 1, 512, 64, 1, 0),
    ('fwd', 300, 64, 5632, 1, 0),
    ('fwd', 100, 1024, 5632, 1, 0),
    ('fwd', 1500, 64, 704, 1, 0),
    ('fwd', 100, 1024, 1408, 1, 0),
    ('fwd', 1, 64, 11264, 1, 1),
    ('fwd', 1, 1024, 2816, 1, 1),
    ('fwd', 1, 64, 64, 1, 1),
    ('fwd', 1, 512, 64, 1, 1),
    ('fwd', 300, 64, 5632, 1, 1),
    ('fwd', 100, 1024, 5632, 1, 1),
    ('fwd', 1500, 64, 704, 1, 1),
    ('fwd', 100, 1024, 1408, 1, 1),
]
