"""The bounded waits of the operators around the feed-forward block: a withheld
arrival ends in the timeout status, no fault, and the context stays usable."""

import pytest

import tensor_core_dense_fp16_gb300 as tc
import test_experts_gpu as experts
import test_residual_norm_gpu as norms
from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu


def times_out(call):
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    tc.hgemm_set_wait_timeout(50_000_000)   # 50 ms per wait
    tc.hgemm_debug_inject(tc.HGEMM_INJECT_DROP_ARRIVAL)
    try:
        call()
        assert tc.hgemm_device_status() == tc.HGEMM_ERR_TIMEOUT
        assert tc.hgemm_device_status() == tc.HGEMM_OK  # the word was cleared by the read
    finally:
        tc.hgemm_debug_inject(tc.HGEMM_INJECT_NONE)
        tc.hgemm_set_wait_timeout(0)


@pytest.mark.parametrize("m,d", [(40, 264), (5, 8192), (2000, 1024)])
@pytest.mark.parametrize("kind", [tc.HGEMM_NORM_RMS, tc.HGEMM_NORM_LAYER])
def test_norms_backward(m, d, kind):
    torch = torch_cuda()
    h = lambda: torch.zeros(m, d, dtype=torch.float16, device="cuda")  # noqa: E731
    gamma, stats = torch.ones(d, dtype=torch.float16, device="cuda"), torch.ones(4, m, device="cuda")
    dz, dh, z, y, dx, dy = (h() for _ in range(6))
    work = torch.empty(tc.hgemm_residual_norm_backward_workspace_size(m, d), dtype=torch.uint8, device="cuda")
    times_out(lambda: tc.hgemm_residual_norm_backward(dz, d, dh, d, z, d, y, d, 1.0, None, kind, gamma, None, kind,
                                                      gamma, stats, dx, d, dy, d, None, None, None, None, None, work, m,
                                                      d))
    norms.run_backward(m, d)


@pytest.mark.parametrize("m,d,f,e,k", [(1, 256, 512, 8, 2), (16, 128, 264, 3, 3), (64, 512, 4104, 4, 4)])
def test_experts(m, d, f, e, k):
    torch = torch_cuda()
    h = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    x, wr, w1, w2, y = h(m, d), h(e, d), h(e, 2 * f, d), h(e, d, f), h(m, d)
    work = torch.empty(tc.hgemm_experts_workspace_size(m, d, f, e, k), dtype=torch.uint8, device="cuda")
    times_out(lambda: tc.hgemm_experts(x, d, wr, d, w1, d, None, w2, f, None, 3, True, k, True, None, 0, y, d, None,
                                       None, work, m, d, f, e))
    experts.run(m, d, f, e, k)
