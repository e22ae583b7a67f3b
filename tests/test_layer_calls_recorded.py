"""Host side of the layer operators on calls whose launches are written down
instead of run: what is refused, what is launched and what workspace is held."""

import os

import pytest

import layer_record as rec

OK, INVALID, OOM = 0, 1, 4


@pytest.fixture(scope="module")
def call(tmp_path_factory):
    if not os.path.exists(rec.CXX):
        pytest.skip("ROCm clang++ not available")
    exe = rec.build(tmp_path_factory.mktemp("record"))
    return lambda *lines: rec.calls(exe, lines)


@pytest.mark.parametrize("line", ["ln 0 40 0 null bias y8", "fwd 0 40 72 null bias res act=1 z8", "fwd 0 40 72 null act=2 z",
                                  "dx 0 40 72 null act=1 z8 actout", "dx 0 40 72 null act=2 z actout add", "dx 0 40 72 null",
                                  "enc 0 40 0 null", "dec 0 40 0 null"])
def test_no_rows_is_no_call(call, line):
    """A batch without rows is taken, with the null addresses of empty tensors,
    whatever the optional arguments, and enqueues nothing."""
    r, = call(line)
    assert r["status"] == OK and r["launches"] == [], r


@pytest.mark.parametrize("line", ["dw 0 40 72 null db", "dw 0 40 72 null x8 db acc", "lngrad 0 40 0 null add"])
def test_no_rows_still_writes_parameter_gradients(call, line):
    r, = call(line)
    assert r["status"] == OK and len(r["launches"]) == 1, r


@pytest.mark.parametrize("line", ["dx 4 40 72 act=1", "dx 4 40 72 actout", "dx 0 40 72 act=7", "dx 0 40 72 act=1 null pad=-1"])
def test_missing_pre_activation_is_refused(call, line):
    r, = call(line)
    assert r["status"] == INVALID and r["launches"] == [], r


@pytest.mark.gpu
def test_empty_tensors_with_an_activation():
    import torch

    import newton_schulz_matrix_step_amd as nsm
    h = nsm.muon_init(0)
    try:
        def e(n):
            return torch.empty(0, n, device="cuda", dtype=torch.bfloat16)

        w = torch.ones(40, 72, device="cuda", dtype=torch.bfloat16)
        for z in (e(40), nsm.Act8.empty(0, 40)):
            nsm.muon_linear_grad_input(h, e(72), w, e(40), act="gelu", z=z, act_out=e(40), add=e(40))
        nsm.muon_linear_forward(h, e(40), w, e(72), act="gelu", z_out=nsm.Act8.empty(0, 72))
        nsm.muon_act_encode(h, e(40), nsm.Act8.empty(0, 40))
        nsm.muon_act_decode(h, nsm.Act8.empty(0, 40), e(40))
        torch.cuda.synchronize()
    finally:
        nsm.muon_destroy(h)


MIB = 1 << 20


def _needs(call, lines):
    """What each call allocates on a handle of its own."""
    cmds = []
    for s in lines:
        cmds += ["new", s]
    return [r["workspace"] for r in call(*cmds)]


# 8-bit layer inputs decoded in the workspace: 2 rows x in bytes, from small to past 256 MiB
GROWING = [f"dw {r} 8192 8192 x8 db" for r in range(1000, 100001, 1000)]


def test_growing_calls_hold_a_bounded_workspace(call):
    """Batches that grow a little at a time: what the handle holds stays under
    four times the largest need (plus the rounding of each block to a MiB), at
    every call, and only a few blocks are ever allocated."""
    need = _needs(call, GROWING)
    held = [r["workspace"] for r in call(*GROWING)]
    assert max(need) > 1024 * MIB and need == sorted(need)
    for n, b in zip(need, held):
        assert n <= b <= 4 * n + 32 * MIB
    assert len(set(held)) <= 12
    # smaller calls afterwards, in any order, allocate nothing
    again = call(*GROWING, *reversed(GROWING))
    assert again[-1]["workspace"] == held[-1]


def test_growth_falls_back_to_the_size_needed(call):
    """Where twice the largest block cannot be allocated, the call's own size is."""
    lines = [f"dw {r} 8192 8192 x8" for r in (20000, 24000)]
    n = _needs(call, lines)
    a, b = call(lines[0], f"limit {n[1]}", lines[1])
    assert a["status"] == OK and b["status"] == OK and a["workspace"] == n[0] and b["workspace"] == sum(n)
    a, b = call(lines[0], f"limit {n[1] - MIB}", lines[1])
    assert b["status"] == OOM and b["launches"] == [] and b["workspace"] == n[0]


def test_capture_finds_a_block_or_is_refused(call):
    big, small = "dw 20000 8192 8192 x8", "dw 10000 8192 8192 x8"
    a, = call(small + " capture")
    assert a["status"] == INVALID and a["launches"] == [] and a["workspace"] == 0
    a, b, c = call(small, small + " capture", big + " capture")
    assert (a["status"], b["status"], c["status"]) == (OK, OK, INVALID) and c["workspace"] == a["workspace"]
    a, b = call(big, small + " capture")
    assert b["status"] == OK and b["workspace"] == a["workspace"]


# Calls whose natural grid has 2^32 threads or more, which no launch can have:
# many rows of a narrow product, 8-bit checkpoints and operands of tens of GB.
WIDE_GRIDS = ["fwd 2147482000 8 8", "fwd 1073741824 8 8 oi", "fwd 2147482624 16 8 f32", "dx 2147482000 8 8",
              "dx 1073741825 16 24 f32 z8 act=1 actout", "fwd 8 8 1048576 bias", "dw 64 1048576 262016", "fwd 2147482000 37 40", "dw 2147483647 7 9 db f32",
              "enc 16777216 4104 0", "enc 33554432 4104 0", "enc 16777217 8192 0 f32", "dec 33554432 4104 0",
              "enc 2147483647 32 0", "dec 2147483647 1 0", "ln 2147483647 8 0 y8", "lngrad 2147483647 64 0 add"]


@pytest.mark.parametrize("line", WIDE_GRIDS)
def test_launches_stay_under_2_32_threads(call, line):
    r, = call(line)
    assert r["status"] == OK and r["launches"], r
    for k in r["launches"]:
        assert 0 < k["grid"] * k["block"] < 2 ** 32, k


@pytest.mark.parametrize("line", ["fwd 2147483647 8 8", "fwd 2147482625 8 8", "dx 1073741825 1048576 8", "dw 8 1048576 1048576",
                                  "ln 8388608 16392 0", "lngrad 8388608 16392 0", "ln 9223372036854775807 20000 0",
                                  "enc 9223372036854775807 20000 0", "fwd 9223372036854775807 8 8"])
def test_more_than_a_launch_can_take_is_refused(call, line):
    r, = call(line)
    assert r["status"] == INVALID and r["launches"] == [], r


def test_checkpoint_slices_cover_every_row(call):
    """A checkpoint pass in several launches: workgroups of one row each, as many as rows."""
    for op in ("enc", "dec"):
        r, = call(f"{op} 33554433 4104 0")
        assert len(r["launches"]) > 1 and sum(k["grid"] for k in r["launches"]) == 33554433
        r, = call(f"{op} 16384 4096 0")
        assert [k["grid"] for k in r["launches"]] == [8192]


@pytest.mark.parametrize("line,streams", [("ln 16 768 0", False), ("ln 2048 768 0 bias y8", False), ("ln 8192 2048 0", False),
                                          ("ln 8193 2048 0", True), ("ln 8192 4096 0 bias", True), ("ln 4096 2048 0 f32", False),
                                          ("ln 8191 2048 0 f32 y8", True), ("ln 5000 12288 0", True), ("ln 9001 4095 0", None),
                                          ("ln 70000 1024 0 shift=1", None)])
def test_only_outputs_past_the_caches_are_streamed(call, line, streams):
    """A norm's output is what the next product reads: it is stored past the L2s
    only where they could not hold it (None: rows without whole 16-byte runs, by element)."""
    r, = call(line)
    k, = r["launches"]
    words = k["kernel"].strip("()").replace(">", "").split(", ")
    assert words[-1] == ("true" if streams else "false"), k
    assert words[1] == ("false" if streams is None else "true"), k
