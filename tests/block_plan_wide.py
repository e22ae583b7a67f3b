"""Gated products of wide layers and long sums that block_plan.CASES leaves out, one for
every kernel that the plan picks there, and the sizes that between them ask for all."""

import math
import random

WIDTHS = (64, 128, 256, 352, 512, 704, 768, 1024, 1280, 1408, 1536, 1792, 2048, 2304, 2560, 2816, 4096, 5120, 5632, 6144,
          7168, 8192, 10240, 11264, 13824, 14336, 16384, 20480, 28672)
ROWS = (1, 8, 64, 100, 200, 300, 512, 700, 1024, 1500, 2048, 3000, 4096, 6000, 8192, 12000, 16384)
KINDS = [(k, dt, lay) for k in ("fwd", "dh", "dx", "dw") for dt in (0, 1) for lay in (0, 1)]


def sweep(seed=1):
    """Every pair of model widths, and sizes of any value spread over their logarithms."""
    out = [(k, r, i, f, dt, lay) for k, dt, lay in KINDS for r in ROWS for i in WIDTHS for f in WIDTHS if r * i * f < 1e12]
    rng = random.Random(seed)

    def size(most):
        return round(math.exp(rng.uniform(0, math.log(most))))

    for k, dt, lay in KINDS:
        drawn = ((size(65536), size(32768), size(32768)) for _ in range(8000))
        out += [(k, r, i, f, dt, lay) for r, i, f in drawn if r * i * f < 1e12]
    return out


# product, rows, in (dh: out), hidden, type, layout
CASES = [
    ("fwd", 100, 5120, 1792, 0, 0),
    ("fwd", 100, 5120, 1792, 0, 1),
    ("fwd", 300, 16384, 10240, 0, 0),
    ("fwd", 300, 14336, 10240, 0, 1),
    ("fwd", 200, 5120, 5632, 0, 1),
    ("dh", 100, 6144, 20480, 0, 0),
    ("dh", 100, 6144, 20480, 0, 1),
    ("dh", 100, 8192, 6144, 0, 0),
    ("dh", 100, 8192, 6144, 0, 1),
    ("dh", 300, 28672, 20480, 0, 0),
    ("dh", 700, 28672, 11264, 0, 1),
    ("dh", 200, 10240, 11264, 0, 0),
    ("dh", 200, 12288, 11264, 0, 1),
    ("dx", 700, 12288, 8192, 0, 0),
    ("dx", 700, 12288, 8192, 0, 1),
]
