"""Products that between them reach every kernel the library's plan can pick:
which product, type and weight layout, where the operands come from, tile edge,
ring depth, split sums or not.  One line each, in the words of the recorded host
build (layer_record.py); sizes end inside tiles in both directions."""

import itertools

POOL = [1, 8, 40, 64, 100, 136, 200, 264, 304, 520, 776, 1000, 1032, 1408, 2000, 2056, 3000, 4104, 8200, 14344]


def sweep():
    """Lines over a wide range of sizes, for every product, type, layout and source."""
    out = []
    for op in ("fwd", "dx", "dw"):
        for words in itertools.product(("", "f32"), ("", "oi"), ("", "shift=1"), ("", "x8") if op == "dw" else ("",)):
            most = 4e10 if "f32" in words else 6e10
            tail = " ".join(w for w in words if w)
            for r, a, b in itertools.product(POOL, POOL, POOL):
                if r * a * b <= most:
                    out.append(f"{op} {r} {a} {b} {tail}".strip())
    return out


def product(call):
    """The product's launch among those of a recorded call."""
    k, = [v for v in call["launches"] if "linear_tile_kernel" in v["kernel"] or "linear_pp_kernel" in v["kernel"]]
    return k


def variant(line, call):
    """The kernel that a recorded call's product runs."""
    k = product(call)
    codes = k["codes"] and not k["a_ld"]
    dma_a, dma_b = k["a_dma"] or k["a_ld"] > 0, k["b_dma"] or k["b_ld"] > 0
    src = ("codes" if dma_b else "codes, any") if codes else "aligned" if dma_a and dma_b else "any"
    ring = bool(k["deep"]) if src == "aligned" and k["tile"] < 256 else None
    words = line.split()
    return words[0], "f32" if "f32" in words else "bf16", "oi" in words, src, k["tile"], ring, k["splits"] > 1


CASES = [
    "dw 776 2000 3000", "dw 776 136 14344", "dw 14344 136 776", "dw 776 14344 520", "dw 2000 14344 264",
    "dw 776 100 8200", "dw 8200 200 264", "dw 776 100 100", "dw 14344 136 200", "dw 1 136 14344 shift=1",
    "dw 100 100 100", "dw 8200 100 136 shift=1", "dw 776 14344 136 x8", "dw 8200 1032 136 x8", "dw 776 3000 136 x8",
    "dw 8200 200 264 x8", "dw 1 136 14344 shift=1 x8", "dw 100 100 100 shift=1 x8", "dw 1000 100 100 shift=1 x8",
    "dw 776 2000 3000 oi", "dw 776 136 14344 oi", "dw 14344 136 776 oi", "dw 776 14344 520 oi",
    "dw 2000 14344 264 oi", "dw 776 100 8200 oi", "dw 8200 200 264 oi", "dw 776 100 100 oi", "dw 14344 136 200 oi",
    "dw 1 136 14344 oi shift=1", "dw 100 100 100 oi", "dw 8200 100 136 oi shift=1", "dw 776 14344 136 oi x8",
    "dw 8200 1032 136 oi x8", "dw 776 3000 136 oi x8", "dw 8200 200 264 oi x8", "dw 1 136 14344 oi shift=1 x8",
    "dw 100 100 100 oi shift=1 x8", "dw 1000 100 100 oi shift=1 x8", "dw 1408 2000 2000 f32", "dw 304 100 8200 f32",
    "dw 14344 100 136 f32", "dw 304 100 100 f32", "dw 2056 136 776 f32", "dw 40 100 100 f32 shift=1",
    "dw 304 100 100 f32 shift=1", "dw 304 2000 136 f32 x8", "dw 14344 100 136 f32 x8", "dw 40 100 100 f32 shift=1 x8",
    "dw 304 100 100 f32 shift=1 x8", "dw 1408 2000 2000 f32 oi", "dw 304 100 8200 f32 oi", "dw 14344 100 136 f32 oi",
    "dw 304 100 100 f32 oi", "dw 2056 136 776 f32 oi", "dw 40 100 100 f32 oi shift=1",
    "dw 304 100 100 f32 oi shift=1", "dw 304 2000 136 f32 oi x8", "dw 14344 100 136 f32 oi x8",
    "dw 40 100 100 f32 oi shift=1 x8", "dw 304 100 100 f32 oi shift=1 x8", "dx 2000 3000 776", "dx 136 14344 776",
    "dx 1000 200 14344", "dx 1032 8200 776", "dx 14344 264 4104", "dx 100 8200 776", "dx 200 264 8200",
    "dx 100 100 776", "dx 136 200 14344", "dx 14344 200 100", "dx 100 8200 304 shift=1", "dx 100 136 14344 shift=1",
    "dx 2000 3000 776 oi", "dx 1032 2056 8200 oi", "dx 136 14344 776 oi", "dx 1000 200 14344 oi",
    "dx 2056 4104 1000 oi", "dx 1000 4104 4104 oi", "dx 100 8200 776 oi", "dx 200 264 8200 oi", "dx 100 100 776 oi",
    "dx 136 200 14344 oi", "dx 14344 200 100 oi shift=1", "dx 100 8200 304 oi shift=1", "dx 100 136 14344 oi shift=1",
    "dx 2000 2000 1408 f32", "dx 100 8200 304 f32", "dx 100 136 14344 f32", "dx 100 100 304 f32",
    "dx 136 776 2056 f32", "dx 100 100 40 f32 shift=1", "dx 100 100 304 f32 shift=1", "dx 2000 2000 1408 f32 oi",
    "dx 100 8200 304 f32 oi", "dx 100 136 14344 f32 oi", "dx 100 100 304 f32 oi", "dx 136 776 2056 f32 oi",
    "dx 100 100 40 f32 oi shift=1", "dx 100 100 304 f32 oi shift=1", "fwd 2000 776 3000", "fwd 1032 8200 2056",
    "fwd 136 776 14344", "fwd 1000 14344 200", "fwd 2056 1000 4104", "fwd 1000 4104 4104", "fwd 100 776 8200",
    "fwd 200 8200 264", "fwd 100 776 100", "fwd 136 14344 200", "fwd 14344 100 200 shift=1",
    "fwd 100 304 8200 shift=1", "fwd 100 14344 136 shift=1", "fwd 2000 776 3000 oi", "fwd 136 776 14344 oi",
    "fwd 1000 14344 200 oi", "fwd 1032 776 8200 oi", "fwd 14344 4104 264 oi", "fwd 100 776 8200 oi",
    "fwd 200 8200 264 oi", "fwd 100 776 100 oi", "fwd 136 14344 200 oi", "fwd 14344 100 200 oi",
    "fwd 100 304 8200 oi shift=1", "fwd 100 14344 136 oi shift=1", "fwd 2000 1408 2000 f32", "fwd 100 304 8200 f32",
    "fwd 100 14344 136 f32", "fwd 100 304 100 f32", "fwd 136 2056 776 f32", "fwd 100 40 100 f32 shift=1",
    "fwd 100 304 100 f32 shift=1", "fwd 2000 1408 2000 f32 oi", "fwd 100 304 8200 f32 oi", "fwd 100 14344 136 f32 oi",
    "fwd 100 304 100 f32 oi", "fwd 136 2056 776 f32 oi", "fwd 100 40 100 f32 oi shift=1",
    "fwd 100 304 100 f32 oi shift=1",
]

# and input gradients that stream act(z) from narrow tiles, or keep it on the widest
STREAMS = ["dx 14344 776 200", "dx 2000 4104 1000"]
