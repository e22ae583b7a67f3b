"""Float64 oracle of the layer operators (layer norm, the linear layer's three
products, 8-bit activation checkpoints), written from their definitions in
``include/muon.h`` and sharing no code with the GPU path.  Each function also
returns, where asked, the sums of magnitudes its rounding-error bounds need."""

from __future__ import annotations

import math

import numpy as np

GROUP = 32


def layernorm(x, gain, bias=None, eps=1e-5):
    """y, mean, rstd of the rows of x."""
    x = np.asarray(x, np.float64)
    mean = x.sum(1) / x.shape[1]
    var = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None] * np.asarray(gain, np.float64)
    return (y if bias is None else y + np.asarray(bias, np.float64)), mean, rstd


def layernorm_grad(dy, x, gain, mean, rstd, add=None):
    """dx, dgain, dbias."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    n = x.shape[1]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    a = dy * np.asarray(gain, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (a - a.sum(1, keepdims=True) / n -
                                                  xh * (a * xh).sum(1, keepdims=True) / n)
    return (dx if add is None else dx + add), (dy * xh).sum(0), dy.sum(0)


def activation(z, kind):
    """(value, derivative)"""
    z = np.asarray(z, np.float64)
    if kind == "gelu":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if kind == "relu_sq":
        r = np.maximum(z, 0.0)
        return r * r, 2 * r
    if kind == "none":
        return z.copy(), np.ones_like(z)
    raise ValueError(kind)


def weight_in_out(w, w_layout):
    w = np.asarray(w, np.float64)
    return w.T if w_layout == "out_in" else w


def linear(x, w, bias=None, act="none", residual=None, w_layout="in_out"):
    """y, z (the pre-activation)"""
    z = np.asarray(x, np.float64) @ weight_in_out(w, w_layout)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = activation(z, act)[0]
    return (y if residual is None else y + np.asarray(residual, np.float64)), z


def linear_grad_input(dy, w, act="none", z=None, add=None, w_layout="in_out"):
    """dx, act(z) (None without z)"""
    dx = np.asarray(dy, np.float64) @ weight_in_out(w, w_layout).T
    v = None
    if z is not None:
        v, d = activation(z, act)
        dx = dx * d
    return (dx if add is None else dx + np.asarray(add, np.float64)), v


def linear_grad_weight(x, dy, w_layout="in_out"):
    """dw as the weight is stored, db"""
    dy = np.asarray(dy, np.float64)
    dw = np.asarray(x, np.float64).T @ dy
    return (dw.T if w_layout == "out_in" else dw), dy.sum(0)


def act8_exponents(x):
    """Exponent byte of every group: the smallest k >= -126 with amax <= 127 * 2^k,
    plus 127; 255 for a group that holds an infinity or a NaN."""
    x = np.abs(np.asarray(x, np.float64))
    r, c = x.shape
    g = -(-c // GROUP)
    out = np.zeros((r, g), np.uint8)
    for i in range(r):
        for j in range(g):
            v = x[i, j * GROUP:(j + 1) * GROUP]
            if not np.all(np.isfinite(v)):
                out[i, j] = 255
                continue
            k = -126
            m = float(v.max())
            if m > 0:
                k = max(-126, math.frexp(m / 127.0)[1])   # m / 127 = f 2^e, 0.5 <= f < 1: 2^e suffices
                if k > -126 and m <= 127.0 * 2.0 ** (k - 1):
                    k -= 1
            out[i, j] = k + 127
    return out


def act8_encode(x):
    """codes, exponents"""
    x = np.asarray(x, np.float64)
    e = act8_exponents(x)
    k = np.repeat(e.astype(np.int64) - 127, GROUP, axis=1)[:, :x.shape[1]]
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.where(k == 128, 0.0, np.rint(x / np.exp2(np.where(k == 128, 0, k).astype(np.float64))))
    return q.astype(np.int8), e


def act8_decode(codes, exps):
    k = np.repeat(np.asarray(exps).astype(np.int64) - 127, GROUP, axis=1)[:, :codes.shape[1]]
    return np.where(k == 128, np.nan, np.asarray(codes, np.float64) * np.exp2(np.minimum(k, 127).astype(np.float64)))
