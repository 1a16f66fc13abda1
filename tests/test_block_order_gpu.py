"""Launches of the block's operators start before the one ahead of them has
ended: what comes before a call on its stream and what comes after keep their
order, on every kernel that starts early (GPU only)."""

import numpy as np
import pytest

import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

HALF_ULP = 2.0 ** -11


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
