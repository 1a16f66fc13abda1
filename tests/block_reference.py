"""The feed-forward block's operators in 64 bits (numpy), from the formulas in
include/hgemm.h, with the error bounds the tests hold the kernels to."""

from __future__ import annotations

import math

import numpy as np

GROUP = 64
ACTS = ("none", "relu", "gelu", "silu", "gelu_erf")

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(u, name):
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "relu":
            return np.where(u < 0, 0.0, u)
        if name == "gelu":
            return 0.5 * u * (1 + np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
        if name == "silu":
            return u / (1 + np.exp(-u))
        if name == "gelu_erf":
            return 0.5 * u * (1 + _erf(u / math.sqrt(2)))
        return u


def act_gradient(u, name):
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "relu":
            return np.where(np.isnan(u), np.nan, (u > 0).astype(np.float64))
        if name == "gelu":
            t = np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))
            return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u * u)
        if name == "silu":
            p = 1 / (1 + np.exp(-u))
            return p * (1 + u * (1 - p))
        if name == "gelu_erf":
            return 0.5 * (1 + _erf(u / math.sqrt(2))) + u * np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
        return np.where(np.isnan(u), np.nan, 1.0)


def kept(codes, scales):
    """The values an 8-bit form stands for; scales [groups][rows]."""
    m, n = codes.shape
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64).T, GROUP, axis=1)[:, :n]


def keep32(x):
    """The 8-bit form of FP32 values, in the header's FP32 operations."""
    m, n = x.shape
    groups = -(-n // GROUP)
    v = np.zeros((m, groups * GROUP), np.float32)
    v[:, :n] = x
    v = v.reshape(m, groups, GROUP)
    top = np.abs(v).max(axis=2)
    top = np.where(np.isnan(v).any(axis=2), np.float32(np.nan), top).astype(np.float32)
    bad = ~np.isfinite(top)
    zero = ~bad & (top < np.float32(2.0 ** -100))
    safe = np.where(bad | zero, np.float32(1), top).astype(np.float32)
    inv = (np.float32(127) / safe).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = np.rint((v * inv[:, :, None]).astype(np.float32))
    q = np.where((bad | zero)[:, :, None], 0, q)
    s = np.where(bad, np.float32(np.nan), np.where(zero, np.float32(0), safe / np.float32(127))).astype(np.float32)
    return q.reshape(m, groups * GROUP)[:, :n].astype(np.int8), np.ascontiguousarray(s.T)


# An FP16 output is rounded once: half a unit in its 11-bit significand, or
# half the smallest subnormal.
def half_rounding(y):
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -25


def product(a, b):
    """a·b in 64 bits (a M×K, b K×N), and a bound on an FP32 accumulation's
    error: at most K/8 + 16 rounded additions, each within 2^-23 of a partial
    sum that is itself at most Σ|a||b|."""
    a, b = a.astype(np.float64), b.astype(np.float64)
    k = a.shape[1]
    return a @ b, 2.0 ** -23 * (k / 8 + 16) * (np.abs(a) @ np.abs(b))


# The activations are 1.13-Lipschitz; their FP32 evaluation (2^x and a
# reciprocal to ~2^-22, a few operations, erf's 2^-23 beside 1) is within
# 2^-19 of |f| + 2^-22, the derivative's within 2^-18.
LIPSCHITZ = 1.13


def act_error(f):
    return 2.0 ** -19 * np.abs(f) + 2.0 ** -22 * (1 + np.abs(f))


def linear(x, w, bias, name, res):
    """(y, its bound, u, its bound)."""
    u, eu = product(x, w.astype(np.float64).T)
    if bias is not None:
        u = u + bias.astype(np.float64)
        eu = eu + 2.0 ** -23 * np.abs(u)
    y = act(u, name)
    ey = LIPSCHITZ * eu + (act_error(y) if name not in ("none", "relu") else 0)
    if res is not None:
        y = y + res.astype(np.float64)
        ey = ey + 2.0 ** -23 * np.abs(y)
    return y, ey + half_rounding(y) * 1.001, u, eu


def dgrad(dy, w, codes, scales, name):
    """(dU, its bound, H, its bound)."""
    g, eg = product(dy, w)
    if codes is None:
        return g, eg + half_rounding(g) * 1.001, None, None
    u = kept(codes, scales)
    h, dh = act(u, name), act_gradient(u, name)
    du = g * dh
    return (du, LIPSCHITZ * eg + 2.0 ** -18 * np.abs(g) + half_rounding(du) * 1.001,
            h, act_error(h) + 2.0 ** -23 * np.abs(u) + half_rounding(h) * 1.001)


def column_sums(dy):
    """Σ rows, and an FP32 sum's bound: at most M/8 + 16 additions in a row."""
    d = dy.astype(np.float64)
    return d.sum(axis=0), 2.0 ** -24 * (d.shape[0] / 8 + 16) * np.abs(d).sum(axis=0) + 1e-30


def layernorm(x, gamma, beta, eps):
    """y, mean, rstd and their bounds: FP32 sums over a row of D values take
    at most D/32 + 32 additions in a row."""
    x = x.astype(np.float64)
    d = x.shape[1]
    mu = x.mean(axis=1)
    c = x - mu[:, None]
    var = (c * c).mean(axis=1)
    rstd = 1 / np.sqrt(var + eps)
    step = 2.0 ** -24 * (d / 32 + 32)
    emu = step * np.abs(x).mean(axis=1) + 1e-30
    # the variance is summed around the computed mean: its relative error is
    # a sum's, plus (emu/σ)²; the root halves it
    ers = rstd * (step + 2.0 ** -22 + (emu * rstd) ** 2)
    xh = c * rstd[:, None]
    y = xh * gamma.astype(np.float64) + beta.astype(np.float64)
    ey = np.abs(gamma.astype(np.float64)) * ((emu * rstd)[:, None] + 2.0 ** -23 * (np.abs(x) * rstd[:, None])
                                             + np.abs(xh) * (ers / rstd + 2.0 ** -22)[:, None])
    return y, ey + 2.0 ** -23 * np.abs(y) + half_rounding(y) * 1.001, mu, emu, rstd, ers


def layernorm_backward(dy, x, gamma, mean, rstd, res):
    """dX, dgamma, dbeta and their bounds."""
    dy, x, gamma = (v.astype(np.float64) for v in (dy, x, gamma))
    mean, rstd = mean.astype(np.float64), rstd.astype(np.float64)
    d, m = x.shape[1], x.shape[0]
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    a, b = g.mean(axis=1, keepdims=True), (g * xh).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (g - a - xh * b)
    step = 2.0 ** -24 * (d / 32 + 32)
    exh = 2.0 ** -22 * ((np.abs(x) + np.abs(mean)[:, None]) * rstd[:, None])  # x̂ in FP32
    ea = step * np.abs(g).mean(axis=1, keepdims=True)
    eb = step * np.abs(g * xh).mean(axis=1, keepdims=True) + (np.abs(g) * exh).mean(axis=1, keepdims=True)
    edx = rstd[:, None] * (ea + np.abs(xh) * eb + exh * np.abs(b)
                           + 2.0 ** -21 * (np.abs(g) + np.abs(a) + np.abs(xh * b)))
    if res is not None:
        dx = dx + res.astype(np.float64)
        edx = edx + 2.0 ** -23 * np.abs(dx)
    esum = 2.0 ** -24 * (m / 8 + 64)
    dgamma, dbeta = (dy * xh).sum(axis=0), dy.sum(axis=0)
    return (dx, edx + half_rounding(dx) * 1.001,
            dgamma, esum * np.abs(dy * xh).sum(axis=0) + (np.abs(dy) * exh).sum(axis=0) + 1e-30,
            dbeta, esum * np.abs(dy).sum(axis=0) + 1e-30)
