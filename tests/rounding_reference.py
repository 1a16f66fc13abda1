"""AdamW's 8-bit states rounded at random (numpy): the random numbers of a
value by its index and the step's number, and the codes that they give."""

from __future__ import annotations

import numpy as np

from around_reference import F32, GROUP

U32 = np.uint32


def mixed(x):
    x = np.asarray(x, U32)
    with np.errstate(over="ignore"):
        x = (x ^ (x >> U32(16))) * U32(0x6A09E667)
        x = (x ^ (x >> U32(15))) * U32(0xBB67AE85)
    return x ^ (x >> U32(16))


_POWERS = np.array([pow(0x9E3779B1, k, 1 << 32) for k in range(8)], U32)


def random_bits(n, step):
    """32 bits for each of a tensor's n values."""
    i = np.arange(n)
    with np.errstate(over="ignore"):
        return mixed((i >> 3).astype(U32) + mixed(step % (1 << 32))) * _POWERS[i & 7]


def _groups(x):
    p = np.zeros(-(-len(x) // GROUP) * GROUP, x.dtype)
    p[:len(x)] = x
    return p.reshape(-1, GROUP)


def _kinds(p):
    """(largest magnitude, whether it is none that can be kept, whether too small)."""
    top = np.abs(p).max(axis=1)
    bad = ~np.isfinite(p).all(axis=1)
    return np.where(bad, F32(1), top).astype(F32), bad, ~bad & (top < F32(2.0 ** -100))


def keep_m(m, step):
    n = len(m)
    p, u = _groups(m), _groups((1 + (2 * (random_bits(n, step) & U32(0xFFF)) + 1.0) / 8192).astype(F32))
    top, bad, zero = _kinds(p)
    safe = np.where(zero, F32(1), top)
    with np.errstate(invalid="ignore"):
        # (a fused product and sum: 48 bits and a number in (1, 2), rounded once; 64 bits
        # round it twice, which tells only within 2^-29 of the middle of two FP32 numbers)
        x = (p.astype(np.float64) * (F32(127) / safe).astype(F32).astype(np.float64)[:, None] + u).astype(F32)
        codes = np.floor(x) - 1
    codes[bad | zero] = 0
    scales = np.where(bad, F32(np.nan), np.where(zero, F32(0), safe / F32(127))).astype(F32)
    return codes.reshape(-1)[:n].astype(np.int8), scales


def keep_v(v, step):
    n = len(v)
    p, u = _groups(v), _groups((random_bits(n, step) >> U32(12)).astype(np.int64))
    top, bad, zero = _kinds(p)
    safe = np.where(zero, F32(1), top)
    with np.errstate(invalid="ignore"):
        r = (p * (F32(1) / safe).astype(F32)[:, None]).astype(F32)
    # eight codes to a doubling, 255 for 1; the lower of two codes is bits >> 20
    codes = (r.view(np.int32).astype(np.int64) - 0x3F800000 + (255 << 20) + u) >> 20
    codes = np.where(r > 0, np.clip(codes, 1, 255), 0)
    codes[bad | zero] = 0
    return (codes.reshape(-1)[:n].astype(np.uint8),
            np.where(bad, F32(np.nan), np.where(zero, F32(0), top)).astype(F32))
