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
