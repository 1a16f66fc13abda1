"""The norms' backward pass over very many narrow rows (GPU only)."""

import ctypes

import pytest

import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import done
from test_residual_norm_gpu import run_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,d", [(320, 1), (321, 1), (4928, 4), (4929, 4), (11000, 3), (15000, 65), (10001, 7)])
@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "none")])
def test_passes(m, d, post, pre):
    run_backward(m, d, post, pre)


@pytest.mark.parametrize("m,d", [(1 << 20, 3), (1 << 20, 1), (1 << 18, 77)])
def test_launches(m, d):
    """A call of very many narrow rows is a few hundred launches at most: at
    least 4608 rows to every three."""
    torch = torch_cuda()
    h = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    x, gamma, stats = [h(m, d) for _ in range(6)], h(d), torch.ones(4, m, device="cuda")
    sums = [torch.full((d,), 7.0, device="cuda") for _ in range(2)]
    work = torch.empty(tc.hgemm_residual_norm_backward_workspace_size(m, d), dtype=torch.uint8, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(keep_graph=True), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        tc.hgemm_residual_norm_backward(x[0], d, x[1], d, x[2], d, x[3], d, 1.0, None, 2, gamma, None, 2, gamma, stats,
                                        x[4], d, x[5], d, None, sums[0], None, sums[1], None, work, m, d)
    nodes = ctypes.c_size_t()
    assert ctypes.CDLL("libcuda.so.1").cuGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None,
                                                       ctypes.byref(nodes)) == 0
    assert 4 <= nodes.value <= 3 * (m // 4608 + 1) + 1
    graph.instantiate()
    graph.replay()
    torch.cuda.synchronize()
    done()
    assert (sums[0] == 0).all() and (sums[1] == 0).all()
