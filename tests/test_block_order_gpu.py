"""Launches of the block's operators start before the one ahead of them has
ended: what comes before a call on its stream and what comes after keep their
order, on every kernel that starts early (GPU only)."""

import numpy as np
import pytest

import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu


# whole numbers small enough that every sum is exact in FP32
def whole(rng, torch, *shape):
    return torch.from_numpy(rng.integers(-2, 3, shape).astype(np.float16)).cuda()


# which product the column sums run beside: several tiles per CTA with room on
# its SMs, few tiles, split K, the turned-around product, odd sizes
@pytest.mark.parametrize("M,N,K", [(256, 8192, 8192), (1024, 2048, 4096), (4096, 640, 1544), (8192, 512, 512),
                                   (4096, 1000, 1000), (1500, 1001, 777)])
def test_sums_beside_their_product(M, N, K):
    torch = torch_cuda()
    rng = np.random.default_rng(M + N + K)
    srcs = [whole(rng, torch, M, N) for _ in range(3)]
    x = whole(rng, torch, M, K)
    wants = [s.double().sum(dim=0) for s in srcs]
    dy, old = torch.empty_like(srcs[0]), whole(rng, torch, N).float()
    dw, db = torch.empty((N, K), dtype=torch.float16, device="cuda"), torch.empty(N, device="cuda")
    got = []
    for i in range(12):
        # written just before, by a copy on the same stream; overwritten just after
        dy.copy_(srcs[i % 3])
        db.copy_(old)
        tc.hgemm_linear_wgrad(dy, N, x, K, dw, K, db, i % 2 == 1, M, N, K)
        got.append(db.clone())
        dy.fill_(float("nan"))
        db.fill_(float("nan"))
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    for i, g in enumerate(got):
        assert torch.equal(g.double(), wants[i % 3] + (old.double() if i % 2 == 1 else 0)), i


# the two kernels that ask L2 for weights ahead of their wait, and the others
@pytest.mark.parametrize("M,N,K", [(1, 1024, 2048), (5, 264, 520), (3, 65, 77), (24, 2048, 2048), (100, 520, 4104),
                                   (40, 2051, 1001), (300, 264, 520), (2048, 2048, 256)])
def test_operands_written_just_before(M, N, K):
    """Weights and rows written by the launch ahead, another value every time."""
    torch = torch_cuda()
    rng = np.random.default_rng(M + N + K)
    xs, ws, bs = ([whole(rng, torch, *s) for _ in range(3)] for s in ((M, K), (N, K), (N,)))
    wants = [x.double() @ w.double().t() + b.double() for x, w, b in zip(xs, ws, bs)]
    x, w, b = (torch.empty_like(t[0]) for t in (xs, ws, bs))
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    got = []
    for i in range(15):
        b.copy_(bs[i % 3])
        # the last launch ahead is the one that writes the rows, or the weights
        for dst, src in ((x, xs), (w, ws))[:: 1 if i % 2 else -1]:
            dst.copy_(src[i % 3])
        tc.hgemm_linear(x, K, w, K, b, tc.HGEMM_ACT_NONE, None, 0, y, N, M, N, K)
        got.append(y.clone())
        x.fill_(float("nan"))
        w.fill_(float("nan"))
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    for i, g in enumerate(got):
        assert torch.equal(g.double(), wants[i % 3].half().double()), i


def test_a_chain_of_early_starts():
    """Each launch's output is the next one's operand, as X, as W and in 8 bits,
    with kernels that start early on both sides."""
    torch = torch_cuda()
    rng = np.random.default_rng(3)
    d = 1024
    f16 = dict(dtype=torch.float16, device="cuda")
    eye = torch.eye(d, **f16)
    q, s = torch.empty((d, d), dtype=torch.int8, device="cuda"), torch.empty((d // 64, d), device="cuda")
    one = torch.ones(d, **f16)
    for i in range(10):
        src = whole(rng, torch, d, d)
        want = torch.layer_norm(src[:8].double(), (d,), eps=1e-5)
        w, back, x, y = (torch.empty((d, d), **f16) for _ in range(4))
        tc.hgemm_linear(src, d, eye, d, None, 0, None, 0, w, d, d, d, d)       # w = src, one wave of tiles
        tc.hgemm_linear(eye, d, w, d, None, 0, None, 0, x, d, 8, d, d)         # 8 rows: x = srcᵀ's first rows
        tc.hgemm_ckpt8_save(w, d, q, d, s, d, d, d)
        tc.hgemm_ckpt8_load(q, d, s, d, 0, back, d, d, d)
        tc.hgemm_layernorm_forward(w, d, one, one - 1, 1e-5, y, d, None, None, 8, d)
        w.fill_(float("nan"))
        assert torch.equal(x[:8], src.t()[:8])
        # (values 0, 1 and 2 of 2: 127, 64 and 0 steps)
        assert (back.double() - src.double()).abs().max() <= 1 / 127
        assert (y[:8].double() - want).abs().max() <= 2.0 ** -9 * want.abs().max()
    assert tc.hgemm_device_status() == tc.HGEMM_OK


@pytest.mark.parametrize("what", ["forward", "backward", "weight"])
def test_few_rows_and_small_weights_time_out(what):
    """The waits of the turned-around product are bounded in all its forms."""
    torch = torch_cuda()
    half = lambda *s: torch.ones(s, dtype=torch.float16, device="cuda")  # noqa: E731
    call = {"forward": lambda: tc.hgemm_linear(half(64, 4096), 4096, half(512, 4096), 4096, None, 2, None, 0,
                                               half(64, 512), 512, 64, 512, 4096),
            "backward": lambda: tc.hgemm_linear_dgrad(half(64, 4096), 4096, half(4096, 512), 512, None, 0, None, 0, 0,
                                                      half(64, 512), 512, None, 0, 64, 4096, 512),
            "weight": lambda: tc.hgemm_linear_wgrad(half(8192, 128), 128, half(8192, 136), 136, half(128, 136), 136, None,
                                                    False, 8192, 128, 136)}[what]
    torch.cuda.synchronize()
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    tc.hgemm_set_wait_timeout(20_000_000)
    tc.hgemm_debug_inject(tc.HGEMM_INJECT_DROP_ARRIVAL)
    try:
        call()
        assert tc.hgemm_device_status() == tc.HGEMM_ERR_TIMEOUT
    finally:
        tc.hgemm_debug_inject(tc.HGEMM_INJECT_NONE)
        tc.hgemm_set_wait_timeout(0)
    call()
    assert tc.hgemm_device_status() == tc.HGEMM_OK
