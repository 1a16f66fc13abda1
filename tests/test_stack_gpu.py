"""Blocks with norms, gates and residual scales around them, their optimizer
and the experts' layer as they are used together, against autograd in 64 bits
(GPU only). An FP16 rounding is 2^-11/√3 = 2.8e-4 of a value in the mean; a
block has at most six in a row each way, and a norm passes a relative error on
as it is: two blocks' twelve are 1.0e-3 in quadrature, held to 4e-3 of a
result's norm. The 8-bit pre-activations (0.6% of u in the mean) move a
gradient by at most a few percent of its norm per block: 5e-2."""

import pytest

import around_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_adamw_gpu import done

pytestmark = pytest.mark.gpu

EPS = 1e-5


def block(g, d, f, act="gelu", norm="rms", beta=False, post="rms", post_beta=False, gate=True, scale=1.0):
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import FeedForward

    def n(*s, scale=1.0, shift=0.0):
        return (torch.randn(*s, generator=g, device="cuda") * scale + shift).half()

    return FeedForward(n(d, scale=0.2, shift=1), n(d, scale=0.1) if beta else None, n(f, d, scale=d ** -0.5),
                       n(f, scale=0.1), n(d, f, scale=f ** -0.5), n(d, scale=0.1), act=act, eps=EPS, norm=norm,
                       post=post, post_gamma=n(d, scale=0.2, shift=1) if post != "none" else None,
                       post_beta=n(d, scale=0.1) if post_beta else None,
                       gate=n(d, scale=0.2, shift=0.5) if gate else None, residual_scale=scale)


def norm64(x, kind, gamma, beta):
    if kind == tc.HGEMM_NORM_LAYER:
        x = x - x.mean(1, keepdim=True)
    x = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * gamma
    return x if beta is None else x + beta


def block64(b, p, x):
    torch = torch_cuda()
    act = {"gelu": lambda u: torch.nn.functional.gelu(u, approximate="tanh"), "silu": torch.nn.functional.silu,
           "relu": torch.relu}[{2: "gelu", 3: "silu", 1: "relu"}[b.act]]
    u = norm64(x, b.norm, p["gamma"], p.get("beta")) @ p["w1"].t() + p["b1"]
    y = act(u) @ p["w2"].t() + p["b2"]
    if b.post != tc.HGEMM_NORM_NONE:
        y = norm64(y, b.post, p["post_gamma"], p.get("post_beta"))
    return b.residual_scale * x + (y if b.gate is None else p["gate"] * y)


def leaves(b):
    return {n: t.double().requires_grad_() for n, t in b.parameters().items()}


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


KINDS = [dict(), dict(norm="layer", beta=True, post="layer", post_beta=True), dict(post="none", scale=0.75),
         dict(norm="layer", post="none", gate=False, scale=1.5), dict(norm="rms", post="none", gate=False),
         dict(norm="rms", beta=True, post="layer", gate=False, act="silu")]


@pytest.mark.parametrize("m,d,f", [(300, 256, 512), (77, 65, 131), (1, 128, 512)])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_a_block(m, d, f, kind):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(kind + m)
    b = block(g, d, f, **KINDS[kind])
    x, dy = (torch.randn(m, d, generator=g, device="cuda").half() for _ in range(2))
    y, saved = b.forward(x)
    grads = b.backward(dy, saved)
    # (a product that keeps nothing may take another kernel, which sums in another order)
    assert off(b(x), y.double()) < 4e-3
    done()
    p, x64 = leaves(b), x.double().requires_grad_()
    want = block64(b, p, x64)
    want.backward(dy.double())
    assert off(y, want.detach()) < 4e-3
    assert off(grads.x, x64.grad) < 5e-2
    assert set(grads.named()) == set(p)
    for n, got in grads.named().items():
        assert off(got, p[n].grad) < 5e-2, n


@pytest.mark.parametrize("m,d,f", [(300, 256, 512), (40, 72, 136), (1000, 1000, 264)])
@pytest.mark.parametrize("last", [dict(), dict(post="none", gate=False), dict(norm="layer", beta=True, post="layer")])
def test_a_stack(m, d, f, last):
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import FeedForwardStack
    g = torch.Generator(device="cuda").manual_seed(m)
    blocks = [block(g, d, f, scale=0.75), block(g, d, f, **last)]
    stack = FeedForwardStack(blocks)
    x, dy = (torch.randn(m, d, generator=g, device="cuda").half() for _ in range(2))
    y, saved = stack.forward(x)
    dx, grads = stack.backward(dy, saved)
    assert off(stack(x), y.double()) < 4e-3
    done()
    ps, x64 = [leaves(b) for b in blocks], x.double().requires_grad_()
    z = x64
    for b, p in zip(blocks, ps):
        z = block64(b, p, z)
    z.backward(dy.double())
    assert off(y, z.detach()) < 4e-3
    assert off(dx, x64.grad) < 5e-2
    for p, gr in zip(ps, grads):
        assert set(gr.named()) == set(p)
        for n, got in gr.named().items():
            assert off(got, p[n].grad) < 5e-2, n
    # and what the blocks give one by one
    z = x
    for b in blocks:
        z = b(z)
    assert off(y, z.double()) < 4e-3


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("master", [True, False])
def test_training_steps(bits, master):
    """Forward, backward and the optimizer, a few steps in a row: each step's
    parameters are the reference's step from the gradients of that step."""
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import AdamW, FeedForwardStack
    from block_reference import half_rounding
    from test_block_gpu import check
    import numpy as np
    g = torch.Generator(device="cuda").manual_seed(9)
    m, d, f = 96, 72, 200
    stack = FeedForwardStack([block(g, d, f), block(g, d, f, norm="layer", beta=True)])
    names = {f"{i}.{n}": t for i, b in enumerate(stack.blocks) for n, t in b.parameters().items()}
    opt = AdamW(names, lr=1e-2, bits=bits, master=master, weight_decay=0.1)
    x, dy = (torch.randn(m, d, generator=g, device="cuda").half() for _ in range(2))
    for step in range(1, 4):
        y, saved = stack.forward(x)
        _, grads = stack.backward(dy, saved)
        by_name = {f"{i}.{n}": t for i, gr in enumerate(grads) for n, t in gr.named().items()}
        num = lambda t: t.detach().cpu().numpy().reshape(-1)  # noqa: E731
        before = [{k: num(v) for k, v in t.items() if hasattr(v, "numel") and k != "grad"} for t in opt.tensors]
        opt.step(by_name, grad_scale=0.5)
        done()
        for name, t, old in zip(opt.names, opt.tensors, before):
            gradient = num(by_name[name])
            if bits == 8:
                ms, vs = ref.kept_m(old["m"], old["m_scales"]), ref.kept_v(old["v"], old["v_scales"])
            else:
                ms, vs = old["m"], old["v"]
            p = old["master"] if master else old["weight"]
            want, bound = ref.adamw(p, gradient, ms, vs, opt.lr, opt.beta1, opt.beta2, opt.eps,
                                    0.1 if t["weight"].dim() > 1 else 0.0, step, 0.5)
            if master:
                check(num(t["master"]), want, bound, name)
                assert np.array_equal(num(t["weight"]), num(t["master"]).astype(np.float16)), name
            else:
                check(num(t["weight"]), want, bound + half_rounding(np.abs(want) + bound) * 1.001, name)


def test_a_training_step_in_a_graph():
    """A captured step, the optimizer's in it, replays to what eager steps give."""
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import AdamW, FeedForwardStack

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(3)
        stack = FeedForwardStack([block(g, 128, 264), block(g, 128, 264)])
        names = {f"{i}.{n}": t for i, b in enumerate(stack.blocks) for n, t in b.parameters().items()}
        x, dy = (torch.randn(200, 128, generator=g, device="cuda").half() for _ in range(2))
        return stack, AdamW(names, lr=1e-3, bits=8), x, dy

    def step(stack, opt, x, dy, dynamic=None):
        y, saved = stack.forward(x)
        dx, grads = stack.backward(dy, saved)
        opt.step({f"{i}.{n}": t for i, gr in enumerate(grads) for n, t in gr.named().items()}, dynamic=dynamic)
        return y, dx

    eager = fresh()
    for _ in range(3):
        want = step(*eager)
    done()
    stack, opt, x, dy = fresh()
    device = torch.zeros(16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(stack, opt, x, dy, device)
    for i in range(1, 4):
        device.copy_(tc.hgemm_adamw_dynamic(opt.lr, 1.0, i))
        graph.replay()
    torch.cuda.synchronize()
    done()
    # lr/(1 − β^t) comes from FP32 on the device and from 64 bits on the host: a unit in the last place of a
    # parameter now and then
    for a, b in zip(got, want):
        assert off(a, b.double()) < 4e-3
    for (n, a), b in zip(zip(opt.names, opt.tensors), eager[1].tensors):
        assert off(a["master"], b["master"].double()) < 1e-4, n


@pytest.mark.parametrize("m", [1, 5, 64, 150])
def test_tokens_through_experts_between_norms(m):
    """What serves a block of experts: the norm in front, the layer, then the norm
    behind with gate and residual and the next block's norm, in one pass."""
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import ExpertFeedForward
    g = torch.Generator(device="cuda").manual_seed(m)
    d, f, e, k = 256, 136, 10, 3
    n = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).half()  # noqa: E731
    layer = ExpertFeedForward(n(e, d, scale=2 * d ** -0.5), n(e, 2 * f, d, scale=d ** -0.5),
                              n(e, d, f, scale=f ** -0.5), k=k)
    x, gate = n(m, d), n(d, scale=0.5)
    g1, g2, g3 = (1 + n(d, scale=0.2) for _ in range(3))
    h, z, nxt = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rms, none = tc.HGEMM_NORM_RMS, tc.HGEMM_NORM_NONE
    tc.hgemm_residual_norm_forward(x, d, 0.0, x, d, None, rms, g1, None, none, None, None, EPS, h, d, None, 0, None, m, d)
    y, chosen, share = layer(h, choices=True)
    tc.hgemm_residual_norm_forward(x, d, 1.0, y, d, gate, rms, g2, None, rms, g3, None, EPS, z, d, nxt, d, None, m, d)
    done()
    h64 = norm64(x.double(), rms, g1.double(), None)
    logits = h.double() @ layer.router.double().t()
    # (up to logits that FP32 sums of these sizes cannot tell apart)
    best = logits.topk(k, dim=1).values
    assert float((logits.gather(1, chosen.long()) - best).abs().max()) < 1e-5
    y64 = torch.zeros_like(h64)
    for j in range(k):
        w1, w2 = layer.w1.double()[chosen[:, j].long()], layer.w2.double()[chosen[:, j].long()]
        u = (w1 @ h64[:, :, None])[:, :, 0]
        y64 += share[:, j:j + 1].double() * (w2 @ (torch.nn.functional.silu(u[:, :f]) * u[:, f:])[:, :, None])[:, :, 0]
    z64 = x.double() + gate.double() * norm64(y64, rms, g2.double(), None)
    assert off(y, y64) < 4e-3 and off(z, z64) < 4e-3
    assert off(nxt, norm64(z64, rms, g3.double(), None)) < 4e-3


def test_a_refused_step_is_not_counted():
    from tensor_core_dense_fp16_gb300.feedforward import AdamW
    torch = torch_cuda()
    p = torch.ones(64, dtype=torch.float16, device="cuda")
    g = torch.full((64,), 0.01, dtype=torch.float16, device="cuda")
    one, other = AdamW({"p": p.clone()}, lr=0.1), AdamW({"p": p.clone()}, lr=0.1)
    for bad in (g[:32], g.double()):
        with pytest.raises((ValueError, TypeError)):
            one.step({"p": bad})
    with pytest.raises(Exception):
        one.step({"p": g}, grad_scale=float("inf"))
    for o in (one, other):
        o.step({"p": g})
        o.step({"p": g})
    done()
    assert one.steps == 2
    assert torch.equal(one.tensors[0]["master"], other.tensors[0]["master"])


def test_parameters_with_other_storage_and_gradients():
    """A parameter whose storage is replaced between steps is stepped where it
    is now; gradients may be of another type at every step."""
    from tensor_core_dense_fp16_gb300.feedforward import AdamW
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(5)
    start = torch.randn(40, 64, generator=g, device="cuda").half()
    grads = [0.01 * torch.randn(40, 64, generator=g, device="cuda") for _ in range(3)]
    grads[1] = grads[1].half()
    p, q, none = start.clone(), start.clone(), torch.empty(0, dtype=torch.float16, device="cuda")
    one = AdamW({"none": none, "p": p}, lr=0.1, bits=8, master=False)
    other = AdamW({"none": none, "p": q}, lr=0.1, bits=8, master=False)
    for grad in grads:
        old = p.data
        p.data = old.clone()
        old.fill_(7)
        one.step({"none": none.clone(), "p": grad})
        other.step({"none": none.clone(), "p": grad.clone()})
        done()
        assert torch.equal(p, q) and (old == 7).all()
    assert not torch.equal(p, start)


def test_layers_are_checked():
    torch = torch_cuda()
    from tensor_core_dense_fp16_gb300.feedforward import AdamW, ExpertFeedForward, FeedForward, FeedForwardStack
    h = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    args = (h(64), h(64), h(128, 64), h(128), h(64, 128), h(64))
    for kw in (dict(post="rms"), dict(post_gamma=h(64)), dict(post_beta=h(64)), dict(norm="none"), dict(gate=h(65))):
        with pytest.raises(ValueError):
            FeedForward(*args, **kw)
    with pytest.raises(ValueError):
        FeedForwardStack([FeedForward(*args), FeedForward(*args, gate=h(64))])
    with pytest.raises(ValueError):
        FeedForwardStack([])
    with pytest.raises(ValueError):
        ExpertFeedForward(h(4, 64), h(4, 256, 64), h(4, 64, 128), k=5)
    with pytest.raises(ValueError):
        ExpertFeedForward(h(4, 64), h(4, 128, 64), h(4, 64, 128), k=2)
    layer = ExpertFeedForward(h(4, 64), h(4, 256, 64), h(4, 64, 128))
    for x, r in ((h(3, 65), None), (h(3, 64), h(2, 64)), (h(64), None)):
        with pytest.raises(ValueError):
            layer(x, r)
    assert layer(h(0, 64)).shape == (0, 64)
    with pytest.raises(ValueError):
        AdamW({"w": h(4)}, lr=1e-3, bits=16)
    with pytest.raises(KeyError):
        AdamW({"w": h(4)}, lr=1e-3).step({})
