"""Float64 oracle of the block operators (gated feed-forward, norms around a block,
dropout), written from their definitions in ``include/muon.h`` and sharing no code
with the GPU path."""

from __future__ import annotations

import math

import numpy as np

from .layer_oracle import weight_in_out


# ---- dropout --------------------------------------------------------------------

def philox4x32(counter, key, rounds=10):
    """The four 32-bit words (lists of Python integers) of one counter and key."""
    x0, x1, x2, x3 = (int(v) for v in counter)
    k0, k1 = (int(v) for v in key)
    for _ in range(rounds):
        p, q = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = (q >> 32) ^ x1 ^ k0, q & 0xFFFFFFFF, (p >> 32) ^ x3 ^ k1, p & 0xFFFFFFFF
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return [x0, x1, x2, x3]


def threshold(p):
    """p * 65536, p rounded to float32 as the library gets it, to nearest (halves to even)."""
    return int(np.rint(np.float64(np.float32(p)) * 65536.0))


def dropout_bits(rows, cols, seed, offset):
    """The 16 bits of every element of a rows x cols matrix."""
    u32, u64 = np.uint64(0xFFFFFFFF), np.uint64
    blocks = -(-cols // 8)
    x0 = np.broadcast_to(np.arange(blocks, dtype=u64)[None, :], (rows, blocks)).copy()
    x1 = np.broadcast_to(np.arange(rows, dtype=u64)[:, None], (rows, blocks)).copy()
    offset %= 2 ** 64
    x2, x3 = np.full_like(x0, offset & 0xFFFFFFFF), np.full_like(x0, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        p, q = x0 * u64(0xD2511F53), x2 * u64(0xCD9E8D57)     # below 2^64
        x0, x1, x2, x3 = (q >> u64(32)) ^ x1 ^ u64(k0), q & u32, (p >> u64(32)) ^ x3 ^ u64(k1), p & u32
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    out = np.empty((rows, blocks, 8), np.int64)
    for i, w in enumerate((x0, x1, x2, x3)):
        out[:, :, 2 * i] = (w & u64(0xFFFF)).astype(np.int64)
        out[:, :, 2 * i + 1] = (w >> u64(16)).astype(np.int64)
    return out.reshape(rows, blocks * 8)[:, :cols]


def dropout_factors(rows, cols, p, seed, offset):
    """What every element is multiplied by: 0 (dropped) or 65536 / (65536 - T)."""
    t = threshold(p)
    keep = dropout_bits(rows, cols, seed, offset) >= t
    return np.where(keep, 65536.0 / (65536 - t) if t < 65536 else 0.0, 0.0)


def dropped(x, factors):
    """x under the mask: 0 where it drops, whatever x is there."""
    return np.where(factors == 0.0, 0.0, np.where(factors == 0.0, 0.0, x) * factors)


# ---- gated feed-forward -----------------------------------------------------------

def gate(z, kind):
    """(value, derivative)"""
    z = np.asarray(z, np.float64)
    if kind == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if kind == "gelu":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    s = 0.5 * (1.0 + np.tanh(0.5 * z))
    if kind == "silu":
        return z * s, s * (1 + z * (1 - s))
    if kind == "sigmoid":
        return s, s * (1 - s)
    raise ValueError(kind)


def gated(x, w_gate, w_up, bias_gate=None, bias_up=None, act="silu", w_layout="in_out"):
    """h, zg, zu"""
    x = np.asarray(x, np.float64)
    zg, zu = x @ weight_in_out(w_gate, w_layout), x @ weight_in_out(w_up, w_layout)
    zg = zg if bias_gate is None else zg + bias_gate
    zu = zu if bias_up is None else zu + bias_up
    return gate(zg, act)[0] * zu, zg, zu


def gated_grad_hidden(dy, w_down, zg, zu, act="silu", w_layout="in_out"):
    """dzg, dzu, h, dh"""
    dh = np.asarray(dy, np.float64) @ weight_in_out(w_down, w_layout).T
    a, d = gate(zg, act)
    return dh * zu * d, dh * a, a * zu, dh


def gated_grad_input(dzg, dzu, w_gate, w_up, add=None, w_layout="in_out"):
    dx = np.asarray(dzg, np.float64) @ weight_in_out(w_gate, w_layout).T
    dx = dx + np.asarray(dzu, np.float64) @ weight_in_out(w_up, w_layout).T
    return dx if add is None else dx + add


# ---- norms around a block -----------------------------------------------------------

def norm(x, kind, eps):
    """(normalised rows, mean, 1 / root); RMS: mean 0"""
    x = np.asarray(x, np.float64)
    mean = x.sum(1) / x.shape[1] if kind == "layer" else np.zeros(x.shape[0])
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).sum(1) / x.shape[1] + eps)
    return (x - mean[:, None]) * rstd[:, None], mean, rstd


def _affine(x, gain, bias):
    x = x if gain is None else x * gain
    return x if bias is None else x + bias


def junction_stream(x, branch, post="none", post_gain=None, post_bias=None, gate=None, alpha=1.0, beta=1.0, factors=1.0,
                    eps=1e-5):
    """s before its rounding, and the branch norm's mean and 1 / root"""
    t, mean, rstd = (np.asarray(branch, np.float64), None, None) if post == "none" else norm(branch, post, eps)
    t = _affine(t, post_gain, post_bias)
    t = t if np.isscalar(factors) else dropped(t, factors)
    t = t if gate is None else t * gate
    return alpha * np.asarray(x, np.float64) + beta * t, mean, rstd


def junction_norm(s, pre, pre_gain=None, pre_bias=None, eps=1e-5):
    """y, mean, 1 / root of the stream s"""
    xh, mean, rstd = norm(s, pre, eps)
    return _affine(xh, pre_gain, pre_bias), mean, rstd


def _norm_grad(a, xh, rstd, kind):
    n = a.shape[1]
    shift = a.sum(1, keepdims=True) / n if kind == "layer" else 0.0
    return rstd[:, None] * (a - shift - xh * ((a * xh).sum(1, keepdims=True) / n))


def junction_grad(dx_stats, dy=None, ds=None, s=None, branch=None, post="none", post_gain=None, post_bias=None, gate=None,
                  pre="none", pre_gain=None, alpha=1.0, beta=1.0, factors=1.0):
    """Every gradient, by name; dx_stats: the norms' statistics by name."""
    r = {}
    g = 0.0 if ds is None else np.asarray(ds, np.float64)
    if pre != "none":
        xh = (s - dx_stats.get("pre_mean", np.zeros(s.shape[0]))[:, None]) * dx_stats["pre_rstd"][:, None]
        g = g + _norm_grad(dy if pre_gain is None else dy * pre_gain, xh, dx_stats["pre_rstd"], pre)
        r["dpre_gain"], r["dpre_bias"] = (dy * xh).sum(0), dy.sum(0)
    r["dx"] = alpha * g
    if branch is None:
        return r
    e = beta * (g if np.isscalar(factors) else dropped(g, factors))
    eg = e if gate is None else e * gate
    if post == "none":
        oh, r["dbranch"] = branch, eg
    else:
        mean = dx_stats.get("post_mean", np.zeros(branch.shape[0]))
        oh = (branch - mean[:, None]) * dx_stats["post_rstd"][:, None]
        r["dbranch"] = _norm_grad(eg if post_gain is None else eg * post_gain, oh, dx_stats["post_rstd"], post)
        r["dpost_gain"], r["dpost_bias"] = (eg * oh).sum(0), eg.sum(0)
    r["dgate"] = (e * _affine(oh, post_gain, post_bias)).sum(0)
    return r
