"""Pins of the block operators' float64 oracle: the generator's published answers,
values worked out by hand, limits, and every gradient against central differences
of its forward function."""

import math

import numpy as np
import pytest

from oracle import block_oracle as bo
from oracle import layer_oracle as lo


@pytest.mark.parametrize("counter,key,want", [
    # the known answers that the generator was published with (Random123, ten rounds)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(bo.philox4x32(counter, key)) == want


def test_dropout_bits_are_the_blocks_halves():
    seed, offset = 0x0123456789ABCDEF, (7 << 32) + 5
    bits = bo.dropout_bits(5, 21, seed, offset)
    assert bits.shape == (5, 21)
    for r, c in ((0, 0), (0, 7), (1, 8), (4, 20), (3, 13)):
        w = bo.philox4x32((c // 8, r, 5, 7), (0x89ABCDEF, 0x01234567))[(c // 2) % 4]
        assert bits[r, c] == (w >> 16 if c % 2 else w & 0xFFFF)
    assert (bo.dropout_bits(5, 21, seed, offset + 2 ** 64) == bits).all()


def test_dropout_probability_and_limits():
    assert bo.threshold(0.5) == 32768 and bo.threshold(0.0) == 0 and bo.threshold(1.0) == 65536
    assert bo.threshold(1.5 / 65536) == 2 and bo.threshold(2.5 / 65536) == 2      # halves to even
    f = bo.dropout_factors(400, 500, 0.1, 3, 4)
    t = bo.threshold(0.1)
    # 200000 draws: the dropped share within 5 standard deviations of T / 65536
    assert abs((f == 0).mean() - t / 65536) < 5 * math.sqrt(0.1 * 0.9 / 200000)
    assert set(np.unique(f)) == {0.0, 65536 / (65536 - t)}
    assert (bo.dropout_factors(3, 9, 0.0, 1, 2) == 1).all() and (bo.dropout_factors(3, 9, 1.0, 1, 2) == 0).all()
    x = np.array([[np.nan, np.inf, 2.0]])
    assert bo.dropped(x, np.array([[0.0, 0.0, 2.0]])).tolist() == [[0.0, 0.0, 4.0]]


def test_gates_by_hand():
    z = np.array([0.0, 1.0, -1.0])
    s1 = 1 / (1 + math.exp(-1))
    assert bo.gate(z, "silu")[0] == pytest.approx([0, s1, s1 - 1], abs=1e-15)
    assert bo.gate(z, "silu")[1] == pytest.approx([0.5, s1 * (2 - s1), (1 - s1) * (1 - s1)], abs=1e-15)
    assert bo.gate(z, "sigmoid")[1] == pytest.approx([0.25, s1 * (1 - s1), s1 * (1 - s1)], abs=1e-15)
    assert bo.gate(z, "relu")[0].tolist() == [0, 1, 0] and bo.gate(z, "relu")[1].tolist() == [0, 1, 0]
    assert bo.gate(z, "gelu")[0] == pytest.approx(lo.activation(z, "gelu")[0])


def test_gated_by_hand():
    x, wg, wu = np.array([[1.0, 2.0]]), np.array([[3.0], [-1.0]]), np.array([[0.5], [0.25]])
    h, zg, zu = bo.gated(x, wg, wu, np.array([2.0]), np.array([1.0]), "relu")
    assert (zg[0, 0], zu[0, 0], h[0, 0]) == (3.0, 2.0, 6.0)
    assert bo.gated(x, wg.T, wu.T, np.array([2.0]), np.array([1.0]), "relu", "out_in")[0][0, 0] == 6.0


def test_norms_by_hand():
    x = np.array([[1.0, -3.0, 2.0, 4.0]])
    xh, mean, rstd = bo.norm(x, "rms", 0.0)
    assert mean[0] == 0 and rstd[0] == pytest.approx(1 / math.sqrt(30 / 4)) and xh[0, 1] == pytest.approx(-3 / math.sqrt(7.5))
    xh, mean, rstd = bo.norm(x, "layer", 0.5)
    assert mean[0] == 1.0 and rstd[0] == pytest.approx(1 / math.sqrt(26 / 4 + 0.5)) and xh[0, 0] == 0
    s, _, _ = bo.junction_stream(np.array([[10.0, 20.0]]), np.array([[3.0, 4.0]]), "rms", np.array([2.0, 1.0]), None,
                                 np.array([0.5, 3.0]), 0.5, 0.25, np.array([[2.0, 0.0]]), 0.0)
    assert s[0] == pytest.approx([5 + 0.25 * 0.5 * 2 * 2 * 3 / math.sqrt(12.5), 10])


def _differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid", "relu"])
@pytest.mark.parametrize("lay", ["in_out", "out_in"])
def test_gated_gradients_by_differences(act, lay):
    rng = np.random.default_rng(5)
    r, i, f, o = 3, 4, 5, 2
    t = (lambda w: w.T.copy()) if lay == "out_in" else (lambda w: w)
    x, wg, wu, wd = rng.normal(size=(r, i)), t(rng.normal(size=(i, f))), t(rng.normal(size=(i, f))), t(rng.normal(size=(f, o)))
    bg, bu, dy = rng.normal(size=f), rng.normal(size=f), rng.normal(size=(r, o))

    def loss(x=x, wg=wg, wu=wu, bg=bg, bu=bu):
        return float((bo.gated(x, wg, wu, bg, bu, act, lay)[0] @ lo.weight_in_out(wd, lay) * dy).sum())

    h, zg, zu = bo.gated(x, wg, wu, bg, bu, act, lay)
    dzg, dzu, h2, _ = bo.gated_grad_hidden(dy, wd, zg, zu, act, lay)
    assert np.allclose(h, h2)
    assert bo.gated_grad_input(dzg, dzu, wg, wu, None, lay) == pytest.approx(_differences(lambda v: loss(x=v), x), rel=1e-6, abs=1e-8)
    for dz, w, k in ((dzg, wg, "wg"), (dzu, wu, "wu")):
        dw, db = lo.linear_grad_weight(x, dz, lay)
        assert dw == pytest.approx(_differences(lambda v: loss(**{k: v}), w), rel=1e-6, abs=1e-8)
        b = {"wg": "bg", "wu": "bu"}[k]
        assert db == pytest.approx(_differences(lambda v: loss(**{b: v}), bg if b == "bg" else bu), rel=1e-6, abs=1e-8)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("full", [True, False])
def test_junction_gradients_by_differences(post, pre, full):
    rng = np.random.default_rng(6)
    r, n, eps = 3, 5, 0.1
    p = {"x": rng.normal(size=(r, n)), "branch": rng.normal(size=(r, n))}
    if full:
        p["gate"] = rng.normal(size=n)
        if post != "none":
            p["post_gain"] = rng.normal(size=n)
        if post == "layer":
            p["post_bias"] = rng.normal(size=n)
        if pre != "none":
            p["pre_gain"] = rng.normal(size=n)
        if pre == "layer":
            p["pre_bias"] = rng.normal(size=n)
    fac = bo.dropout_factors(r, n, 0.3, 11, 12) if full else 1.0
    ds, dy = rng.normal(size=(r, n)), rng.normal(size=(r, n))

    def run(**kw):
        q = {**p, **kw}
        s, pm, pr = bo.junction_stream(q["x"], q["branch"], post, q.get("post_gain"), q.get("post_bias"), q.get("gate"), 0.75,
                                       0.5, fac, eps)
        st = {"post_mean": pm, "post_rstd": pr}
        loss = (s * ds).sum()
        if pre != "none":
            y, m, rs = bo.junction_norm(s, pre, q.get("pre_gain"), q.get("pre_bias"), eps)
            st.update(pre_mean=m, pre_rstd=rs)
            loss += (y * dy).sum()
        return float(loss), s, {k: v for k, v in st.items() if v is not None}

    _, s, st = run()
    g = bo.junction_grad(st, dy, ds, s, p["branch"], post, p.get("post_gain"), p.get("post_bias"), p.get("gate"), pre,
                         p.get("pre_gain"), 0.75, 0.5, fac)
    for k in p:
        want = _differences(lambda v: run(**{k: v})[0], p[k])
        assert g["d" + k] == pytest.approx(want, rel=1e-6, abs=1e-8), k


def test_junction_without_a_branch():
    rng = np.random.default_rng(7)
    s, dy, gain = rng.normal(size=(2, 6)), rng.normal(size=(2, 6)), rng.normal(size=6)
    _, _, rstd = bo.junction_norm(s, "rms", gain, None, 0.1)
    g = bo.junction_grad({"pre_rstd": rstd}, dy, None, s, pre="rms", pre_gain=gain)
    want = _differences(lambda v: float((bo.junction_norm(v, "rms", gain, None, 0.1)[0] * dy).sum()), s)
    assert g["dx"] == pytest.approx(want, rel=1e-6, abs=1e-8) and "dbranch" not in g
