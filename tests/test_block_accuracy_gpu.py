"""Where an FP32 evaluation of the block's formulas can lose its digits: the
activations' tails and rows far from zero (GPU only)."""

import math

import numpy as np
import pytest

import block_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def normal_cdf(u):
    return 0.5 * _erfc(-u / math.sqrt(2))


def density(u):
    return np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)


# u²/2 = 18 at u = -6 is rounded a few times, each 2^-24 of it: e^(−u²/2) is within
# 2^-18.2 of itself (as erfc is, whose argument's rounding moves it by 2x² + 1
# times as much); what multiplies it is good to 2^-20. So within 2^-17 of each
# term.
RELATIVE = 2.0 ** -17


def dev(a):
    return torch_cuda().from_numpy(np.ascontiguousarray(a)).cuda()


# one row, few rows, a batch, one wave of tiles, more, odd sizes
@pytest.mark.parametrize("M,N,K", [(1, 1200, 8), (20, 80, 40), (100, 520, 2056), (300, 264, 72), (2048, 2048, 64),
                                   (33, 65, 77)])
def test_erf_gelu_in_its_tail(M, N, K):
    """U is exactly u: one column of X is u, one of W is 1, or the other way round."""
    torch = torch_cuda()
    count = M if M > 8 else N
    u = np.linspace(-6, -3, count).astype(np.float16)
    x, w = np.zeros((M, K), np.float16), np.zeros((N, K), np.float16)
    x[:, 3], w[:, 3] = (u, 1) if M > 8 else (1, u)
    u = u.astype(np.float64)
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    tc.hgemm_linear(dev(x), K, dev(w), K, None, tc.HGEMM_ACT_GELU_ERF, None, 0, y, N, M, N, K)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    want = u * normal_cdf(u)
    want = want[:, None] if M > 8 else want[None, :]
    err = np.abs(y.cpu().numpy().astype(np.float64) - want)
    assert (err <= RELATIVE * np.abs(want) + ref.half_rounding(want) * 1.001).all(), err.max()


@pytest.mark.parametrize("M,N,K", [(20, 72, 1024), (300, 264, 128), (2048, 64, 2048), (33, 65, 131)])
def test_erf_gelu_gradient_in_its_tail(M, N, K):
    torch = torch_cuda()
    codes = np.broadcast_to(-64 - np.arange(K) % 64, (M, K)).astype(np.int8)
    scales = np.full((-(-K // 64), M), 6 / 127, np.float32)
    u = ref.kept(codes, scales)
    dy, w = np.zeros((M, N), np.float16), np.zeros((N, K), np.float16)
    dy[:, 5], w[5] = 1, 1
    du, h, y = (torch.empty((M, K), dtype=torch.float16, device="cuda") for _ in range(3))
    tc.hgemm_linear_dgrad(dev(dy), N, dev(w), K, dev(codes), K, dev(scales), M, tc.HGEMM_ACT_GELU_ERF, du, K, h, K,
                          M, N, K)
    tc.hgemm_ckpt8_load(dev(codes), K, dev(scales), M, tc.HGEMM_ACT_GELU_ERF, y, K, M, K)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    # (û is one more FP32 product: 2^-24 of u, times the formulas' steepness, at most u² + 1 = 37)
    want = u * normal_cdf(u)
    for got in (h, y):
        err = np.abs(got.cpu().numpy().astype(np.float64) - want)
        assert (err <= 2 * RELATIVE * np.abs(want) + ref.half_rounding(want) * 1.001).all(), err.max()
    terms = normal_cdf(u), u * density(u)
    want = terms[0] + terms[1]
    err = np.abs(du.cpu().numpy().astype(np.float64) - want)
    assert (err <= 2 * RELATIVE * (np.abs(terms[0]) + np.abs(terms[1])) + ref.half_rounding(want) * 1.001).all()


def norm_backward_bounds(dy, x, gamma, mean, rstd, res):
    """block_reference's values; bounds for x̂ = (x − mean)·rstd in FP32, whose
    rounding is relative to x̂ itself: the difference is rounded once, the
    product once, whatever the row's distance from zero."""
    d, m = x.shape[1], x.shape[0]
    dx, _, dgamma, _, dbeta, edb = ref.layernorm_backward(dy, x, gamma, mean, rstd, res)
    dy, x, gamma, mean, rstd = (v.astype(np.float64) for v in (dy, x, gamma, mean, rstd))
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    a, b = g.mean(axis=1, keepdims=True), (g * xh).mean(axis=1, keepdims=True)
    step = 2.0 ** -24 * (d / 32 + 32)
    exh = 2.0 ** -23 * np.abs(xh)
    ea = step * np.abs(g).mean(axis=1, keepdims=True)
    eb = step * np.abs(g * xh).mean(axis=1, keepdims=True) + (np.abs(g) * exh).mean(axis=1, keepdims=True)
    edx = rstd[:, None] * (ea + np.abs(xh) * eb + exh * np.abs(b) + 2.0 ** -21 * (np.abs(g) + np.abs(a) + np.abs(xh * b)))
    if res is not None:
        edx = edx + 2.0 ** -23 * np.abs(dx)
    edg = 2.0 ** -24 * (m / 8 + 64) * np.abs(dy * xh).sum(axis=0) + (np.abs(dy) * exh).sum(axis=0) + 1e-30
    return dx, edx + ref.half_rounding(dx) * 1.001, dgamma, edg, dbeta, edb


# every group size of the ring, and the rows that it does not take
@pytest.mark.parametrize("D", [264, 1024, 2048, 4096, 8192, 16384, 1001, 20000])
@pytest.mark.parametrize("center,spread", [(3000.0, 2.0), (40000.0, 32.0), (1000.0, 0.0), (60000.0, 0.0)])
def test_norm_backward_of_rows_far_from_zero(D, center, spread):
    """Rows whose values differ by a few units of a large FP16 number, or not at all (x̂ is 0)."""
    torch = torch_cuda()
    M = 9
    rng = np.random.default_rng(D)
    x = (center + spread * rng.integers(-2, 3, (M, D))).astype(np.float16)
    gamma = (1 + 0.2 * rng.standard_normal(D)).astype(np.float16)
    dy, r = (0.1 * rng.standard_normal((2, M, D))).astype(np.float16)
    x64 = x.astype(np.float64)
    mean = x64.mean(axis=1).astype(np.float32)
    rstd = (1 / np.sqrt(x64.var(axis=1) + 1e-5)).astype(np.float32)
    dx = torch.empty((M, D), dtype=torch.float16, device="cuda")
    dg, db = (torch.empty(D, device="cuda") for _ in range(2))
    ws = torch.empty(tc.hgemm_layernorm_backward_workspace_size(M, D), dtype=torch.uint8, device="cuda")
    tc.hgemm_layernorm_backward(dev(dy), D, dev(x), D, dev(gamma), dev(mean), dev(rstd), dev(r), D, dx, D, dg, db, ws,
                                M, D)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    want = norm_backward_bounds(dy, x, gamma, mean, rstd, r)
    for got, value, bound, what in zip((dx, dg, db), want[::2], want[1::2], ("dx", "dgamma", "dbeta")):
        err = np.abs(got.cpu().numpy().astype(np.float64) - value)
        assert (err <= bound).all(), (what, err.max(), np.broadcast_to(bound, err.shape)[err > bound][0])
