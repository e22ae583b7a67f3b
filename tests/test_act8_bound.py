"""How far an element of an 8-bit checkpoint may be off, against its group's
largest magnitude: the bound that include/muon.h states, reached and not passed."""

import os

import numpy as np

from oracle import layer_oracle as lo

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muon.h")


def _worst(x):
    """Largest error of the groups (rows) of x, relative to each group's largest magnitude."""
    e = np.abs(lo.act8_decode(*lo.act8_encode(x)) - x).max(1)
    return e / np.abs(x).max(1)


def test_bound_is_stated_reached_and_kept():
    text = open(HEADER).read()
    text = " ".join(text[:text.index("typedef struct muon_act8")].replace("*", " ").split())
    assert "1/127 of its group's largest magnitude (1/254 at best)" in text
    x = np.zeros((2, 32))
    # a largest magnitude just over 63.5 takes step 1: a tie is half of that off
    x[0, :2] = 63.5 * (1 + 2.0 ** -20), 0.5
    # at 127 steps the same half step is 1/254 of it
    x[1, :2] = 127.0, 0.5
    w = _worst(x)
    assert 1 / 128 < w[0] <= 1 / 127 and w[1] == 1 / 254
    rng = np.random.default_rng(9)
    r = rng.standard_normal((4000, 32)) * np.exp2(rng.uniform(-100, 100, (4000, 1)))
    assert _worst(r).max() <= 1 / 127


def test_groups_at_the_smallest_step():
    """Up to 63.5 of the smallest step, 2^-126, an element is off by at most half of it, however small it is."""
    s = 2.0 ** -126
    x = np.array([[63.5 * s, 0.5 * s] + [0.25 * s] * 30, [0.5 * s] * 32])
    q, e = lo.act8_encode(x)
    assert (e == 1).all()
    assert np.abs(lo.act8_decode(q, e) - x).max() <= s / 2
    assert _worst(x)[1] == 1.0      # a group of nothing but half a step is lost
