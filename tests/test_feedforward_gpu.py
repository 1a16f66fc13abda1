"""The feed-forward block as it is used: a training step and single tokens,
against 64 bits (GPU only). An FP16 rounding is 2^-11/√3 = 2.8e-4 of a value
in the mean; a result here has at most five of them in a row, in quadrature
6.3e-4, held to 2e-3 of the result's norm. Against the block without 8-bit
pre-activations (a step of max|u|/127 over 64 values, 0.6% of them in the
mean) the gradients are held to 2e-2."""

import numpy as np
import pytest

import block_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu


def make(m, d, f, act, seed):
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import FeedForward
    rng = np.random.default_rng(seed)
    p = {"gamma": 1 + 0.2 * rng.standard_normal(d), "beta": 0.1 * rng.standard_normal(d),
         "w1": rng.standard_normal((f, d)) / d ** 0.5, "b1": 0.1 * rng.standard_normal(f),
         "w2": rng.standard_normal((d, f)) / f ** 0.5, "b2": 0.1 * rng.standard_normal(d)}
    p = {k: v.astype(np.float16) for k, v in p.items()}
    x, dy = rng.standard_normal((m, d)).astype(np.float16), (0.1 * rng.standard_normal((m, d))).astype(np.float16)
    block = FeedForward(**{k: torch.from_numpy(v).cuda() for k, v in p.items()}, act=act)
    return block, {k: v.astype(np.float64) for k, v in p.items()}, x, dy


def reference(p, x, dy, act, u_kept=None):
    """(y, gradients) in 64 bits; u_kept: pre-activations to go back through."""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    h, _, mu, _, rstd, _ = ref.layernorm(x, p["gamma"], p["beta"], 1e-5)
    u = h @ p["w1"].T + p["b1"]
    y = x + ref.act(u, act) @ p["w2"].T + p["b2"]
    u = u if u_kept is None else u_kept
    a = ref.act(u, act)
    du = (dy @ p["w2"]) * ref.act_gradient(u, act)
    dx, _, dgamma, _, dbeta, _ = ref.layernorm_backward(du @ p["w1"], x, p["gamma"], mu, rstd, dy)
    return y, {"x": dx, "gamma": dgamma, "beta": dbeta, "w1": du.T @ h, "b1": du.sum(axis=0), "w2": dy.T @ a,
               "b2": dy.sum(axis=0)}


def off(got, want):
    return np.linalg.norm(got.detach().cpu().numpy().astype(np.float64) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("m,d,f,act", [(300, 256, 1024, "gelu"), (1000, 264, 520, "silu"), (77, 65, 131, "gelu_erf"),
                                       (1, 128, 512, "gelu"), (2048, 512, 2048, "gelu")])
def test_training_step(m, d, f, act):
    torch = torch_cuda()
    block, p, x, dy = make(m, d, f, act, seed=m + d)
    y, saved = block.forward(torch.from_numpy(x).cuda())
    grads = block.backward(torch.from_numpy(dy).cuda(), saved)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    kept = ref.kept(saved.codes.cpu().numpy(), saved.scales.cpu().numpy())
    want_y, same_u = reference(p, x, dy, act, kept)
    _, exact_u = reference(p, x, dy, act)
    assert off(y, want_y) < 2e-3
    for name, want in same_u.items():
        assert off(getattr(grads, name), want) < 2e-3, name
        assert off(getattr(grads, name), exact_u[name]) < 2e-2, name


def test_tokens_one_by_one_are_the_prompt():
    torch = torch_cuda()
    block, p, x, dy = make(40, 256, 1024, "gelu", seed=5)
    dx = torch.from_numpy(x).cuda()
    y, _ = block.forward(dx)
    want, _ = reference(p, x, dy, "gelu")
    for rows in (1, 5, 17):
        for i in range(0, 40, rows):
            got = block(dx[i:i + rows].contiguous())
            assert off(got, want[i:i + rows]) < 2e-3
    assert off(block(dx), want) < 2e-3
    assert tc.hgemm_device_status() == tc.HGEMM_OK


def test_no_tokens():
    torch = torch_cuda()
    block, _, _, _ = make(1, 64, 256, "gelu", seed=6)
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    y, saved = block.forward(x)
    g = block.backward(x, saved)
    assert y.shape == (0, 64) and g.x.shape == (0, 64)
    for t in (g.gamma, g.beta, g.w1, g.b1, g.w2, g.b2):
        assert (t == 0).all()


def test_step_in_a_graph():
    """A captured step replays to the same bits as an eager one."""
    torch = torch_cuda()
    block, _, x, dy = make(300, 256, 1024, "gelu", seed=7)
    dx, ddy = torch.from_numpy(x).cuda(), torch.from_numpy(dy).cuda()

    def step():
        y, saved = block.forward(dx)
        return y, block.backward(ddy, saved)

    y0, g0 = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y1, g1 = step()
    graph.replay()
    torch.cuda.synchronize()
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    assert torch.equal(y0, y1)
    for name in ("x", "gamma", "beta", "w1", "b1", "w2", "b2"):
        assert torch.equal(getattr(g0, name), getattr(g1, name)), name


def test_shapes_are_checked():
    block, _, _, _ = make(1, 64, 256, "gelu", seed=8)
    torch = torch_cuda()
    with pytest.raises(ValueError):
        block(torch.zeros((3, 65), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        type(block)(block.gamma, block.beta, block.w2, block.b1, block.w2, block.b2)
    with pytest.raises(KeyError):
        type(block)(block.gamma, block.beta, block.w1, block.b1, block.w2, block.b2, act="tanh")
