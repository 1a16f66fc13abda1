"""What the experts' layer keeps of h between its two products (GPU only).

The sums here are exact: x and the one weight of a row of W1 are FP16 numbers
in [1, 2), so that h = x·w has 22 bits and lies in [1, 4); W2 is the unit
matrix, the one expert chosen has share e^0/e^0 = 1, and the residual is −h
rounded to FP16. What is left, at most 2^-10 and a multiple of 2^-20, is an
FP16 number: it is Y to the bit where h's 22 bits are kept, and 0 where h was
rounded to FP16's 11."""

import numpy as np
import pytest

import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_experts_gpu import call

pytestmark = pytest.mark.gpu


def layer(m, d, e, gated, seed):
    """The values of `call`, token i for expert i % e, and h."""
    rng = np.random.default_rng(seed)
    one_to_two = lambda *s: (1 + rng.integers(0, 1024, s) / 1024).astype(np.float16)  # noqa: E731
    x, w = one_to_two(m, d), one_to_two(e, d)
    expert = np.arange(m) % e
    wr = np.zeros((e, d), np.float16)
    wr[:, :e] = 64 * np.eye(e)
    x[np.arange(m), expert] = 1.9990234375  # the largest of its row's first e
    x[:, :e][np.arange(e) != expert[:, None]] = 1
    w1 = np.zeros((e, 2 * d if gated else d, d), np.float16)
    if gated:  # (g, u) = (x·w, x·w/x[last]): f(g)·u with u = 1, from a row that picks a column of ones
        x[:, d - 1] = 1
        w1[:, d:, d - 1] = 1
    w1[:, np.arange(d), np.arange(d)] = w
    w2 = np.broadcast_to(np.eye(d, dtype=np.float16), (e, d, d)).copy()
    h = x.astype(np.float64) * w[expert].astype(np.float64)
    return {"x": x, "wr": wr, "w1": w1, "w2": w2, "b1": None, "b2": None, "r": -h.astype(np.float16)}, h, expert


# one, two and four tiles of eight tokens to a read of the weights; rows that
# 16-byte accesses describe and others; F in one run and in two
@pytest.mark.parametrize("m,e", [(1, 4), (5, 8), (12, 3), (24, 2), (32, 2), (40, 1), (64, 1), (64, 3)])
@pytest.mark.parametrize("d,pad,offset", [(64, 0, 0), (136, 3, 1), (77, 0, 0), (1032, 0, 0)])
@pytest.mark.parametrize("gated", [False, True])
def test_h_keeps_its_22_bits(m, e, d, pad, offset, gated):
    v, h, expert = layer(m, d, e, gated, m + d)
    y, chosen, share = call(v, "none", gated, 1, True, pad=pad, offset=offset)
    assert (chosen[:, 0] == expert).all() and (share == 1).all()
    left = h + v["r"].astype(np.float64)
    assert (left != 0).any() and (left == left.astype(np.float16)).all()
    assert (y == left.astype(np.float16)).all()


@pytest.mark.parametrize("m,e", [(3, 2), (24, 2), (64, 1)])
def test_h_past_fp16_is_infinite_and_a_nan_is_a_nan(m, e):
    v, _, expert = layer(m, 64, e, False, 3)
    v["r"] = None
    v["x"][0, 10], v["x"][1, 20], v["x"][2, 30] = 60000, -60000, np.nan
    v["w1"][:, np.arange(64), np.arange(64)] = 1.5
    v["w2"][:] = 2.0 ** -10  # (every output sums its token's h)
    y, chosen, _ = call(v, "none", False, 1, True)
    assert (y[0] == np.inf).all() and (y[1] == -np.inf).all() and np.isnan(y[2]).all()
    assert (chosen[[0, 1], 0] == expert[:2]).all()
    want = (v["x"].astype(np.float64)[3:] * 1.5).sum(axis=1) * 2.0 ** -10
    # (64 values of at most 11 bits by 1.5, below 2^8 in all: exact, rounded once)
    assert (y[3:] == want.astype(np.float16)[:, None]).all()
    assert torch_cuda().cuda.is_available() and tc.hgemm_device_status() == tc.HGEMM_OK


@pytest.mark.parametrize("d,f", [(136, 264), (77, 131)])
def test_a_token_is_the_same_in_any_company(d, f):
    """One expert, so that F is cut alike for any number of tokens: pairs of
    rows in one tile, in two and in four give the same sums."""
    from test_experts_gpu import make
    v = make(64, d, f, 1, True, False, True, seed=5)
    all_y = call(v, "silu", True, 1, True)[0]
    for m in (1, 3, 4, 5, 8, 9, 16, 17, 33):
        y = call({**v, "x": v["x"][:m], "r": v["r"][:m]}, "silu", True, 1, True)[0]
        assert (y == all_y[:m]).all(), m
