"""Host-side checks of the block operators' binding, without a GPU: struct layouts
and codes against the header, and the shapes, dtypes, names and devices the binding
refuses before anything reaches the library."""

import ctypes
import os
import subprocess

import pytest
import torch

import newton_schulz_matrix_step_amd as nsm
from newton_schulz_matrix_step_amd import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = ("muon_gated_args", "muon_gated_grad_hidden_args", "muon_gated_grad_input_args", "muon_gated_grad_weight_args",
           "muon_dropout_mask", "muon_dropout_args", "muon_blocknorm_args", "muon_blocknorm_grad_args")


def test_struct_layouts_match_header(tmp_path):
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
    for prefix, table in (("MUON_GATE_", nsm.GATES), ("MUON_NORM_", nsm.NORMS)):
        for k, v in table.items():
            assert f"{prefix}{k.upper()} = {v}" in text


def b16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def q8(r, c):
    return nsm.Act8.empty(r, c, "cpu")


def refuses(f, cases):
    for args, kw, what in cases:
        with pytest.raises(ValueError, match=what):
            f(0, *args, **kw)


def test_binding_refuses_gated_arguments():
    x, w, h = b16(4, 8), b16(8, 6), b16(4, 6)
    refuses(nsm.muon_gated_forward, [
        ((x, w, w, b16(4, 5)), {}, "h has shape"),
        ((x, w, b16(8, 7), h), {}, "w_up has shape"),
        ((x, w, w.float(), h), {}, "w_up is"),
        ((x, w, w, h), {"w_layout": "out_in"}, "x has shape"),
        ((x, w, w, h), {"act": "swish"}, "act must be"),
        ((x, w, w, h), {"bias_up": b16(7)}, "bias_up has shape"),
        ((x, w, w, h), {"bias_gate": b16(6), "bias_up": torch.zeros(6)}, "bias_up is"),
        ((x, w, w, h), {"gate_out": h}, "both"),
        ((x, w, w, h), {"gate_out": h, "up_out": q8(4, 6)}, "both"),
        ((x, w, w, h), {"gate_out": q8(4, 6), "up_out": q8(4, 5)}, "up_out has shape"),
        ((x, w, b16(8, 12)[:, :6], h), {}, "one leading dimension"),
        ((x.half(), w, w, h), {}, "bfloat16 or float32"),
        ((x, w, w, h), {}, "GPU"),
    ])
    refuses(nsm.muon_gated_grad_hidden, [
        ((x, b16(6, 8), h, h, h, b16(4, 5)), {}, "dup has shape"),
        ((x, b16(6, 8), h, q8(4, 6), h, h), {}, "both"),
        ((x, b16(6, 8), None, h, h, h), {}, "both"),
        ((x, b16(6, 7), h, h, h, h), {}, "dy has shape"),
        ((x, b16(6, 8), h, h, h, h), {"h_out": torch.zeros(4, 6)}, "h_out is"),
        ((x, b16(6, 8), h, h, h, b16(4, 8)[:, :6]), {}, "one leading dimension"),
    ])
    refuses(nsm.muon_gated_grad_input, [
        ((h, h, w, w, b16(4, 7)), {}, "dx has shape"),
        ((h, b16(4, 7), w, w, x), {}, "dup has shape"),
        ((h, h, w, w, x), {"add": b16(3, 8)}, "add has shape"),
        ((h, h, w, w, x), {}, "GPU"),
    ])
    refuses(nsm.muon_gated_grad_weight, [
        ((b16(5, 8), h, h, w, w), {}, "x has shape"),
        ((q8(4, 7), h, h, w, w), {}, "x has shape"),
        ((x, h, h, w, w.float()), {}, "dw_up is"),
        ((x, h, h, w, w), {"db_up": b16(5)}, "db_up has shape"),
    ])


def test_binding_refuses_dropout_arguments():
    with pytest.raises(ValueError, match="p must lie"):
        nsm.Dropout(1.5, 0)
    with pytest.raises(ValueError, match="p must lie"):
        nsm.Dropout(float("nan"), 0)
    with pytest.raises(ValueError, match="step must be"):
        nsm.Dropout(0.5, 0, step=torch.zeros(1))
    d = nsm.Dropout(0.5, -1, 2 ** 64 + 3)
    assert d._c(None).seed == 2 ** 64 - 1 and d._c(None).offset == 3
    x = b16(4, 8)
    refuses(nsm.muon_dropout, [
        ((x, b16(4, 7), d), {}, "y has shape"),
        ((x, torch.zeros(4, 8), d), {}, "y is"),
        ((x, x, d), {"add": b16(3, 8)}, "add has shape"),
        ((x, x, d), {}, "GPU"),
    ])


def test_binding_refuses_block_norm_arguments():
    x, g = b16(4, 8), b16(8)
    refuses(nsm.muon_blocknorm_forward, [
        ((x,), {"y": b16(4, 7), "pre_norm": "rms"}, "y has shape"),
        ((x,), {"y": x, "pre_norm": "batch"}, "pre_norm must be"),
        ((x,), {"branch": x, "s": torch.zeros(4, 8)}, "s is"),
        ((x,), {"branch": x, "s": x, "gate": b16(7)}, "gate has shape"),
        ((x,), {"branch": x, "s": x, "pre_gain": g, "gate": torch.zeros(8)}, "gate is"),
        ((x,), {"y": x, "pre_norm": "rms", "pre_rstd": b16(4)}, "pre_rstd must be float32"),
        ((x,), {"y": x, "pre_norm": "rms", "y8": q8(4, 9)}, "y8 has shape"),
        ((x[0],), {}, "2-D"),
        ((x,), {"y": x, "pre_norm": "rms"}, "GPU"),
    ])
    refuses(nsm.muon_blocknorm_backward, [
        ((x,), {"ds": torch.zeros(4, 8)}, "ds is"),
        ((x,), {"dy": x, "s": b16(3, 8), "pre_norm": "rms"}, "s has shape"),
        ((x,), {"dy": x, "branch": torch.zeros(4, 8)}, "branch is"),
        ((x,), {"dy": x, "pre_gain": g, "dpre_gain": torch.zeros(8)}, "dpre_gain is"),
        ((x,), {"dy": x, "pre_gain": b16(16)[::2]}, "contiguous"),
    ])


def test_a_pair_of_one_row_may_have_two_leading_dimensions():
    k = _abi._Args("t", b16(1, 8))
    assert _abi._pair(k, ("a", "b"), b16(1, 8), b16(1, 16)[:, :8], (1, 8), torch.bfloat16, "x")[2] >= 8
