"""The operators around the feed-forward block in 64 bits (numpy), from the
formulas in include/hgemm.h, with the error bounds the tests hold the kernels
to: the norms around a block, AdamW, and the experts' layer."""

from __future__ import annotations

import numpy as np

from block_reference import LIPSCHITZ, act, act_error, half_rounding, keep32, kept, product

NORMS = ("none", "layer", "rms")


def row_step(d):
    """An FP32 sum over a row of d values takes at most d/32 + 32 additions in
    a row, each within 2^-24 of a partial sum."""
    return 2.0 ** -24 * (d / 32 + 32)


def norm(v, ev, kind, gamma, beta, eps):
    """(n, its bound, μ, its bound, ρ, its bound) of rows v known to within ev."""
    d = v.shape[1]
    step = row_step(d)
    if kind == "layer":
        mu = v.mean(axis=1, keepdims=True)
        emu = step * np.abs(v).mean(axis=1, keepdims=True) + ev.mean(axis=1, keepdims=True) + 1e-30
    else:
        mu = emu = np.zeros((v.shape[0], 1))
    c = v - mu
    ec = ev + emu + 2.0 ** -23 * (np.abs(v) + np.abs(mu))
    power = (c * c).mean(axis=1, keepdims=True)
    # Σc² with each c off by ec: 2·|c|·ec + ec², and a sum's own error; a mean
    # that is off adds its square. The root halves a relative error.
    epower = step * power + (2 * np.abs(c) * ec + ec * ec).mean(axis=1, keepdims=True)
    rho = 1 / np.sqrt(power + eps)
    erho = rho * (0.5 * epower / (power + eps) + 2.0 ** -22)
    # (beyond first order where the error is a large part of the row's power)
    erho = erho + rho * (epower / (power + eps)) ** 2
    n = c * rho * gamma + (0 if beta is None else beta)
    en = np.abs(gamma) * (ec * (rho + erho) + np.abs(c) * erho + 2.0 ** -22 * np.abs(c) * rho) + 2.0 ** -23 * np.abs(n)
    return n, en, mu[:, 0], emu[:, 0], rho[:, 0], erho[:, 0]


def double(x):
    return None if x is None else x.astype(np.float64)


def residual_norm(x, alpha, y, gate, post, post_gamma, post_beta, pre, pre_gamma, pre_beta, eps):
    """{name: (value, bound)} of z, h and the statistics."""
    x, y, gate, pg, pb, qg, qb = map(double, (x, y, gate, post_gamma, post_beta, pre_gamma, pre_beta))
    out = {}
    n, en = y, np.zeros_like(y)
    if post != "none":
        n, en, mu, emu, rho, erho = norm(y, en, post, pg, pb, eps)
        out["post_mean"], out["post_rstd"] = (mu, emu), (rho, erho)
    w = 1.0 if gate is None else gate
    z = alpha * x + w * n
    ez = np.abs(w) * en + 2.0 ** -22 * (np.abs(alpha * x) + np.abs(w * n))
    out["z"] = z, ez + half_rounding(np.abs(z) + ez) * 1.001
    if pre != "none":
        h, eh, mu, emu, rho, erho = norm(z, ez, pre, qg, qb, eps)
        out["pre_mean"], out["pre_rstd"] = (mu, emu), (rho, erho)
        out["h"] = h, eh + half_rounding(np.abs(h) + eh) * 1.001
    return out


def residual_norm_backward(dz_in, dh, z, y, alpha, gate, post, post_gamma, post_beta, pre, pre_gamma, stats):
    """{name: (value, bound)} of dx, dy and the vectors' gradients. The bounds
    cover b1 and b2 summed from dz as well as from the sums of its terms."""
    dz_in, dh, z, y, gate, pg, pb, qg, stats = map(double, (dz_in, dh, z, y, gate, post_gamma, post_beta, pre_gamma,
                                                            stats))
    m, d = y.shape
    step = row_step(d)
    esum = 2.0 ** -24 * (m / 8 + 64)
    mean = lambda v: v.mean(axis=1, keepdims=True)  # noqa: E731
    out = {}
    dz = np.zeros((m, d)) if dz_in is None else dz_in
    terms, edz = np.abs(dz), np.zeros((m, d))
    if pre != "none":
        mu, rho = stats[2][:, None], stats[3][:, None]
        zh = (z - mu) * rho
        ezh = 2.0 ** -22 * (np.abs(z) + np.abs(mu)) * rho
        g = dh * qg
        a1 = mean(g) if pre == "layer" else np.zeros((m, 1))
        ea1 = step * mean(np.abs(g)) if pre == "layer" else 0
        a2 = mean(g * zh)
        ea2 = 2 * step * mean(np.abs(g * zh)) + mean(np.abs(g) * ezh)
        dz = dz + rho * (g - a1 - zh * a2)
        terms = terms + rho * (np.abs(g) + np.abs(a1) + np.abs(zh * a2))
        edz = rho * (ea1 + np.abs(zh) * ea2 + ezh * np.abs(a2)) + 2.0 ** -21 * terms
        out["dpre_gamma"] = ((dh * zh).sum(axis=0), esum * np.abs(dh * zh).sum(axis=0)
                             + (np.abs(dh) * ezh).sum(axis=0) + 1e-30)
        out["dpre_beta"] = dh.sum(axis=0), esum * np.abs(dh).sum(axis=0) + 1e-30
    dx = alpha * dz
    out["dx"] = dx, abs(alpha) * edz + 2.0 ** -23 * np.abs(dx) + half_rounding(np.abs(dx) + abs(alpha) * edz) * 1.001
    w = np.ones(d) if gate is None else gate
    yh, eyh = y, np.zeros_like(y)
    if post != "none":
        mu, rho = stats[0][:, None], stats[1][:, None]
        yh = (y - mu) * rho
        eyh = 2.0 ** -22 * (np.abs(y) + np.abs(mu)) * rho
        wg = w * pg
        b1 = mean(wg * dz) if post == "layer" else np.zeros((m, 1))
        b2 = mean(wg * dz * yh)
        # each term of a sum is off by its own error; the sum's additions are within step of the terms' magnitudes
        eb1 = 4 * step * mean(np.abs(wg) * terms) + mean(np.abs(wg) * edz) if post == "layer" else 0
        eb2 = 4 * step * mean(np.abs(wg * yh) * terms) + mean(np.abs(wg) * (np.abs(yh) * edz + eyh * terms))
        dy = rho * (wg * dz - b1 - yh * b2)
        edy = rho * (np.abs(wg) * edz + eb1 + np.abs(yh) * eb2 + eyh * np.abs(b2)
                     + 2.0 ** -21 * (np.abs(wg * dz) + np.abs(b1) + np.abs(yh * b2)))
    else:
        dy = w * dz
        edy = np.abs(w) * edz + 2.0 ** -23 * np.abs(dy)
    out["dy"] = dy, edy + half_rounding(np.abs(dy) + edy) * 1.001
    s1, s0 = (dz * yh).sum(axis=0), dz.sum(axis=0)
    es1 = esum * np.abs(dz * yh).sum(axis=0) + (np.abs(dz) * eyh + edz * (np.abs(yh) + eyh)).sum(axis=0) + 1e-30
    es0 = esum * np.abs(dz).sum(axis=0) + edz.sum(axis=0) + 1e-30
    if post != "none":
        out["dpost_gamma"] = w * s1, np.abs(w) * (es1 + 2.0 ** -23 * np.abs(s1))
        out["dpost_beta"] = w * s0, np.abs(w) * (es0 + 2.0 ** -23 * np.abs(s0))
        b = np.zeros(d) if pb is None else pb
        out["dgate"] = pg * s1 + b * s0, np.abs(pg) * es1 + np.abs(b) * es0 + 2.0 ** -22 * (np.abs(pg * s1)
                                                                                          + np.abs(b * s0))
    else:
        out["dgate"] = s1, es1
    return out


# ------------------------------------------------------------------------ AdamW

GROUP = 64
F32 = np.float32


def keep_m(m):
    """The 8-bit form of FP32 values one behind the other: (codes, scales)."""
    codes, scales = keep32(m[None, :])
    return codes[0], scales[:, 0].copy()


def kept_m(codes, scales):
    """FP32, as a step reads them."""
    return codes.astype(F32) * np.repeat(scales, GROUP)[:len(codes)]


def keep_v(v):
    """The 8-bit floats of FP32 values that are not negative: (codes, scales)."""
    n = len(v)
    p = np.zeros(-(-n // GROUP) * GROUP, F32)
    p[:n] = v
    p = p.reshape(-1, GROUP)
    top = np.where(np.isnan(p).any(axis=1), F32(np.nan), p.max(axis=1)).astype(F32)
    bad, zero = ~np.isfinite(top), np.isfinite(top) & (top < F32(2.0 ** -100))
    inv = (F32(1) / np.where(bad | zero, F32(1), top)).astype(F32)
    with np.errstate(invalid="ignore", over="ignore"):
        r = (p * inv[:, None]).astype(F32)
    # what 255 − c eighths of a doubling below 1 stand for, the nearest of them
    # (halves up), found by comparison
    value = np.array([0.0] + [2.0 ** ((c - 255) // 8) * (1 + ((c - 255) % 8) / 8) for c in range(1, 256)])
    middle = (value[2:] + value[1:-1]) / 2
    codes = 1 + np.searchsorted(middle, np.where(np.isnan(r), 0, r).astype(np.float64), side="right")
    codes = np.where(r > 0, codes, 0)
    codes[bad | zero] = 0
    scales = np.where(bad, F32(np.nan), np.where(zero, F32(0), top)).astype(F32)
    return codes.reshape(-1)[:n].astype(np.uint8), scales


def kept_v(codes, scales):
    c = codes.astype(np.int64)
    r = np.where(c > 0, 2.0 ** ((c - 255) // 8).astype(np.float64) * (1 + ((c - 255) % 8) / 8), 0).astype(F32)
    return r * np.repeat(scales, GROUP)[:len(codes)]


def adamw_states(g, m, v, beta1, beta2, grad_scale):
    """m and v after the step, FP32 operation by operation."""
    with np.errstate(over="ignore", invalid="ignore"):
        g = (g.astype(F32) * F32(grad_scale)).astype(F32)
        m = (m * F32(beta1)).astype(F32) + (g * F32(1 - beta1)).astype(F32)
        v = (v * F32(beta2)).astype(F32) + ((g * g).astype(F32) * F32(1 - beta2)).astype(F32)
    return m, v


def adamw(p, g, m, v, lr, beta1, beta2, eps, decay, step, grad_scale=1.0):
    """(p, its bound) after the step in 64 bits, from FP32 states before it."""
    p, g, m, v = (x.astype(np.float64) for x in (p, g, m, v))
    g = g * grad_scale
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    # each FP32 state: two products and a sum, their factors rounded too
    em = 2.0 ** -22 * (np.abs(beta1 * m) + np.abs((1 - beta1) * g))
    below = np.sqrt(v1 / (1 - beta2 ** step)) + eps
    update = lr * (m1 / (1 - beta1 ** step)) / below
    # v within 2^-22 and its root half of that; root, reciprocal, three factors and a sum: 2^-20 in all
    e = lr / (1 - beta1 ** step) * em / below + 2.0 ** -19 * np.abs(update)
    new = p - lr * decay * p - update
    return new, e + 2.0 ** -22 * (np.abs(p) + np.abs(update))


# ---------------------------------------------------------------------- experts

def experts(x, wr, w1, b1, w2, b2, name, gated, normalize, res, chosen):
    """(logits, their bound, share, its bound, y, its bound) for the experts
    that the rows chose; w1 E×F×D (2F), w2 E×D×F."""
    x64 = x.astype(np.float64)
    m, k = chosen.shape
    f, d = w2.shape[2], x.shape[1]
    logits, el = product(x64, wr.astype(np.float64).T)
    top = logits.max(axis=1, keepdims=True)
    weight = np.exp(logits - top)
    picked = np.take_along_axis(weight, chosen, axis=1)
    share = picked / (picked if normalize else weight).sum(axis=1, keepdims=True)
    # e^(l − top) and the sum below it, each off by the logits' error (twice) and 2^-20
    eshare = share * (4 * el.max(axis=1, keepdims=True) * 1.01 + 2.0 ** -19)
    y, ey = np.zeros((m, d)), np.zeros((m, d))
    if res is not None:
        y += res.astype(np.float64)
    for i in range(m):
        for j in range(k):
            e = chosen[i, j]
            u, eu = product(x64[i:i + 1], w1[e].astype(np.float64).T)
            if b1 is not None:
                u = u + b1[e].astype(np.float64)
                eu = eu + 2.0 ** -23 * np.abs(u)
            h, eh = act(u[:, :f], name), LIPSCHITZ * eu[:, :f]
            if name not in ("none", "relu"):
                eh = eh + act_error(h)
            if gated:
                up, eup = u[:, f:], eu[:, f:]
                eh = eh * (np.abs(up) + eup) + np.abs(h) * eup + 2.0 ** -23 * np.abs(h * up)
                h = h * up
            eh = eh + half_rounding(np.abs(h) + eh) * 1.001
            wt = w2[e].astype(np.float64).T
            o, eo = product(h, wt)
            eo = eo + (1 + 2.0 ** -20 * f) * (eh @ np.abs(wt))
            if b2 is not None:
                o = o + b2[e].astype(np.float64)
                eo = eo + 2.0 ** -23 * np.abs(o)
            y[i] += share[i, j] * o[0]
            ey[i] += (share[i, j] + eshare[i, j]) * eo[0] + eshare[i, j] * np.abs(o[0]) + 2.0 ** -22 * (
                np.abs(y[i]) + np.abs(share[i, j] * o[0]))
    return logits, el, share, eshare, y, ey + half_rounding(np.abs(y) + ey) * 1.001


__all__ = ["NORMS", "adamw", "adamw_states", "experts", "keep_m", "keep_v", "kept", "kept_m", "kept_v", "residual_norm",
           "residual_norm_backward"]
