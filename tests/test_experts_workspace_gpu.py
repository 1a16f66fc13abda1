"""One workspace for every number of tokens up to a largest batch's (GPU only)."""

import pytest

import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import done
from test_experts_workspace import NARROW

pytestmark = pytest.mark.gpu


def weights(d, f, e, seed):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).half()  # noqa: E731
    return n, 4 * n(e, d), n(e, 2 * f, d), n(e, d, f)


@pytest.mark.parametrize("d,f,e,k", NARROW)
def test_calls_of_1_to_64_tokens(d, f, e, k):
    torch = torch_cuda()
    n, wr, w1, w2 = weights(d, f, e, d + e)
    size = tc.hgemm_experts_workspace_size(64, d, f, e, k)
    work = torch.empty(size + 64, dtype=torch.uint8, device="cuda")
    x = n(64, d) * d ** 0.5
    for m in range(1, 65):
        out = []
        for ws in (work, torch.empty(tc.hgemm_experts_workspace_size(m, d, f, e, k), dtype=torch.uint8, device="cuda")):
            ws.fill_(255)
            y = torch.empty(m, d, dtype=torch.float16, device="cuda")
            tc.hgemm_experts(x, d, wr, d, w1, d, None, w2, f, None, 3, True, k, True, None, 0, y, d, None, None, ws, m,
                             d, f, e, workspace_bytes=min(ws.numel(), size))
            out.append(y)
        assert torch.equal(*out) and (work[size:] == 255).all(), m
    done()


@pytest.mark.parametrize("m", [1, 64, 65, 113, 127, 128, 191])
@pytest.mark.parametrize("d,f,e,k", NARROW[:2])
def test_a_layer_of_any_number_of_rows(m, d, f, e, k):
    """Pieces of 64 rows and a shorter one: each row as by itself."""
    from tensor_core_dense_fp16_gb300.feedforward import ExpertFeedForward
    torch = torch_cuda()
    n, wr, w1, w2 = weights(d, f, e, 7)
    layer = ExpertFeedForward(wr, w1, w2, k=k)
    x = n(m, d) * d ** 0.5
    y, chosen, share = layer(x, residual=x, choices=True)
    done()
    want = x.double()
    for j in range(k):
        a, b = w1[chosen[:, j].long()].double(), w2[chosen[:, j].long()].double()
        u = (a @ x.double()[:, :, None])[:, :, 0]
        want = want + share[:, j:j + 1].double() * (b @ (torch.nn.functional.silu(u[:, :f]) * u[:, f:])[:, :, None])[:, :, 0]
    # one rounding to FP16 and sums in 32 bits
    assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -11
