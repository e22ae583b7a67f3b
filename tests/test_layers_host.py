"""Host-side checks of the layer operators' binding, without a GPU: struct
layouts against the header, and the shapes, dtypes, names and devices the
binding refuses before anything reaches the library."""

import ctypes
import os
import subprocess

import pytest
import torch

import newton_schulz_matrix_step_amd as nsm
from newton_schulz_matrix_step_amd import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ("muon_act8", "muon_layernorm_args", "muon_layernorm_grad_args", "muon_linear_args",
           "muon_linear_grad_input_args", "muon_linear_grad_weight_args")


def test_struct_layouts_match_header(tmp_path):
    """Size and every field's offset of the six structs."""
    body, want = [], []
    for name in STRUCTS:
        st = getattr(_abi, name)
        body.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(st))
        for f, _ in st._fields_:
            body.append(f'printf("%zu\\n", offsetof({name}, {f.rstrip("_")}));')
            want.append(getattr(st, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){' + "".join(body) +
                   "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def test_codes_match_header():
    text = open(os.path.join(ROOT, "include", "muon.h")).read()
    for key, val in (("MUON_ACT_NONE", nsm.ACTIVATIONS["none"]), ("MUON_ACT_GELU", nsm.ACTIVATIONS["gelu"]),
                     ("MUON_ACT_RELU_SQ", nsm.ACTIVATIONS["relu_sq"]), ("MUON_W_IN_OUT", nsm.W_LAYOUTS["in_out"]),
                     ("MUON_W_OUT_IN", nsm.W_LAYOUTS["out_in"])):
        assert f"{key} = {val}" in text
    assert f"#define MUON_ACT8_GROUP {nsm.MUON_ACT8_GROUP}" in text


def b16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_act8_shapes_and_dtypes():
    a = nsm.Act8.empty(3, 65, device="cpu")
    assert tuple(a.codes.shape) == (3, 65) and tuple(a.exponents.shape) == (3, 3) and tuple(a.shape) == (3, 65)
    with pytest.raises(ValueError, match="int8"):
        nsm.Act8(torch.zeros(2, 3), torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        nsm.Act8(torch.zeros(2, 33, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="2-D"):
        nsm.Act8(torch.zeros(6, dtype=torch.int8), torch.zeros(1, dtype=torch.uint8))


def test_binding_refuses_norm_arguments():
    x, g, v = b16(4, 8), b16(8), torch.zeros(4)
    f = nsm.muon_layernorm_forward
    for args, kw, what in [
        ((x, g, None, b16(4, 7)), {}, "y has shape"),
        ((x, b16(7), None, b16(4, 8)), {}, "gain has shape"),
        ((x, g, torch.zeros(8), b16(4, 8)), {}, "bias is"),
        ((x, g, None, torch.zeros(4, 8)), {}, "y is"),
        ((x.half(), g, None, b16(4, 8)), {}, "bfloat16 or float32"),
        ((x, g, None, b16(4, 8)), {"mean": b16(4)}, "mean must be float32"),
        ((x, g, None, b16(4, 8)), {"mean": torch.zeros(5)}, "mean has shape"),
        ((x, g, None, b16(4, 8)), {"y8": nsm.Act8.empty(4, 9, "cpu")}, "y8 has shape"),
        ((x[0], g, None, b16(4, 8)), {}, "2-D"),
        ((x, g, None, b16(4, 8)), {}, "GPU"),
    ]:
        with pytest.raises(ValueError, match=what):
            f(0, *args, **kw)
    with pytest.raises(ValueError, match="dgain is"):
        nsm.muon_layernorm_backward(0, x, x, g, v, v, b16(4, 8), torch.zeros(8))
    with pytest.raises(ValueError, match="add has shape"):
        nsm.muon_layernorm_backward(0, x, x, g, v, v, b16(4, 8), b16(8), add=b16(3, 8))
    with pytest.raises(ValueError, match="vectors must be contiguous"):
        nsm.muon_layernorm_backward(0, x, x, b16(16)[::2], v, v, b16(4, 8), b16(8))


def test_binding_refuses_linear_arguments():
    x, w = b16(4, 8), b16(8, 6)
    for args, kw, what in [
        ((x, w, b16(4, 5)), {}, "y has shape"),
        ((x, w, b16(4, 6)), {"w_layout": "out_in"}, "x has shape"),
        ((x, w, b16(4, 6)), {"w_layout": "io"}, "w_layout must be"),
        ((x, w, b16(4, 6)), {"bias": b16(8)}, "bias has shape"),
        ((x, w.float(), b16(4, 6)), {}, "w is"),
        ((x, w, b16(4, 6)), {"z_out": torch.zeros(4, 6)}, "z_out is"),
        ((x, w, b16(4, 6)), {"z_out": nsm.Act8.empty(4, 8, "cpu")}, "z_out has shape"),
        ((x, w, b16(4, 6)), {"residual": b16(6, 4)}, "residual has shape"),
        ((x, w, b16(4, 6)), {}, "GPU"),
    ]:
        with pytest.raises(ValueError, match=what):
            nsm.muon_linear_forward(0, *args, **kw)
    with pytest.raises(ValueError, match="z has shape"):
        nsm.muon_linear_grad_input(0, b16(4, 6), w, b16(4, 8), act="gelu", z=b16(4, 6))
    with pytest.raises(ValueError, match="dy has shape"):
        nsm.muon_linear_grad_input(0, b16(4, 8), w, b16(4, 8))
    with pytest.raises(ValueError, match="x has shape"):
        nsm.muon_linear_grad_weight(0, b16(5, 8), b16(4, 6), w)
    with pytest.raises(ValueError, match="db has shape"):
        nsm.muon_linear_grad_weight(0, x, b16(4, 6), w, db=b16(8))
    with pytest.raises(ValueError, match="q has shape"):
        nsm.muon_act_encode(0, x, nsm.Act8.empty(4, 9, "cpu"))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        nsm.muon_act_decode(0, nsm.Act8.empty(4, 8, "cpu"), x.half())


def test_binding_refuses_strided_columns():
    with pytest.raises(ValueError, match="unit column stride"):
        _abi._ld2(b16(8, 4).t())
    assert _abi._ld2(b16(1, 8)[:, :4]) == 8 and _abi._ld2(b16(8, 8)[:, :1]) == 8
