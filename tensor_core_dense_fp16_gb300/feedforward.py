"""A transformer's feed-forward block on the library's operators:

    y = x + f(LN(x)·W1ᵀ + b1)·W2ᵀ + b2

trained with its pre-activations kept in 8 bits, and run token by token. All
tensors are CUDA FP16 (statistics, scales and the gradients of vectors FP32);
``w1`` is F×D and ``w2`` D×F, a feature per row.

    block = FeedForward(gamma, beta, w1, b1, w2, b2, act="gelu")
    y, saved = block.forward(x)            # training: x is M×D
    grads = block.backward(dy, saved)      # FeedForwardGradients
    y = block(x)                           # inference: nothing kept

What forward leaves for the backward pass is x itself, two numbers per row and
M×F bytes plus a scale per 64 of them: the norm's output is computed again from
x, and the activation's from the 8-bit pre-activations, by the product that
needs their derivative anyway.

Around it: a norm behind the block, a gate and a residual scale (FeedForward's
own arguments, and FeedForwardStack, which fuses them with the next block's
norm), ExpertFeedForward, the same layer as a mixture of experts for tokens, and
AdamW, which steps all parameters in one launch.
``python -m tensor_core_dense_fp16_gb300.feedforward`` runs a training step with
its optimizer's, and a token through the block and through experts.
"""

from __future__ import annotations

import operator
from dataclasses import dataclass
from typing import Any

import tensor_core_dense_fp16_gb300 as tc

ACTIVATIONS = {"none": tc.HGEMM_ACT_NONE, "relu": tc.HGEMM_ACT_RELU, "gelu": tc.HGEMM_ACT_GELU,
               "silu": tc.HGEMM_ACT_SILU, "gelu_erf": tc.HGEMM_ACT_GELU_ERF}


NORMS = {"none": tc.HGEMM_NORM_NONE, "layer": tc.HGEMM_NORM_LAYER, "rms": tc.HGEMM_NORM_RMS}


@dataclass
class Saved:
    """What the backward pass needs of a forward pass."""
    x: Any
    mean: Any
    rstd: Any
    codes: Any        # M×F signed bytes
    scales: Any       # ⌈F/64⌉×M
    y: Any = None     # the branch's output, where a norm or a gate lies behind it
    stats: Any = None  # the norm behind the branch (rows 0 and 1 of 4×M)


@dataclass
class FeedForwardGradients:
    x: Any
    gamma: Any
    beta: Any
    w1: Any
    b1: Any
    w2: Any
    b2: Any
    post_gamma: Any = None
    post_beta: Any = None
    gate: Any = None

    def named(self):
        """The parameters' gradients by name."""
        return {n: g for n, g in vars(self).items() if n != "x" and g is not None}


class FeedForward:
    def __init__(self, gamma, beta, w1, b1, w2, b2, act: str = "gelu", eps: float = 1e-5, norm: str = "layer",
                 post: str = "none", post_gamma=None, post_beta=None, gate=None, residual_scale: float = 1.0):
        """norm: "layer" or "rms", in front of the block (beta None: 0). post: the
        norm behind it ("none", "layer", "rms"), gate a vector, residual_scale a
        number: y = residual_scale·x + gate ⊙ N_post(branch)."""
        import torch
        self.torch = torch
        self.F, self.D = w1.shape
        for name, t, shape in (("gamma", gamma, (self.D,)), ("beta", beta, (self.D,)), ("w1", w1, (self.F, self.D)),
                               ("b1", b1, (self.F,)), ("w2", w2, (self.D, self.F)), ("b2", b2, (self.D,)),
                               ("post_gamma", post_gamma, (self.D,)), ("post_beta", post_beta, (self.D,)),
                               ("gate", gate, (self.D,))):
            if t is None and name in ("beta", "post_gamma", "post_beta", "gate"):
                continue
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.gamma, self.beta, self.w1, self.b1, self.w2, self.b2 = gamma, beta, w1, b1, w2, b2
        self.act, self.eps = ACTIVATIONS[act], eps
        self.norm, self.post = NORMS[norm], NORMS[post]
        if self.norm == tc.HGEMM_NORM_NONE:
            raise ValueError("norm must be layer or rms")
        if (post_gamma is None) != (self.post == tc.HGEMM_NORM_NONE) or (post_gamma is None and post_beta is not None):
            raise ValueError("post_gamma and post_beta belong to a norm behind the block")
        self.post_gamma, self.post_beta, self.gate, self.residual_scale = post_gamma, post_beta, gate, residual_scale
        # the residual branch of a plain block is the second product's epilogue
        self.plain = self.post == tc.HGEMM_NORM_NONE and gate is None and residual_scale == 1.0
        self.layer = self.norm == tc.HGEMM_NORM_LAYER and beta is not None

    def parameters(self):
        """The block's parameters by name."""
        names = ("gamma", "beta", "w1", "b1", "w2", "b2", "post_gamma", "post_beta", "gate")
        return {n: getattr(self, n) for n in names if getattr(self, n) is not None}

    def _half(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.float16, device=self.w1.device)

    def _float(self, *shape):
        return self.torch.empty(shape, dtype=self.torch.float32, device=self.w1.device)

    def _rows(self, x, name: str):
        if x.dim() != 2 or x.shape[1] != self.D or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous M×{self.D} matrix")
        return x.shape[0]

    def __call__(self, x):
        """The block's output; nothing is kept (a prompt, or one token per row)."""
        return self._run(x, None)

    def _saved(self, x, m):
        return Saved(x, self._float(m), self._float(m),
                     self.torch.empty((m, self.F), dtype=self.torch.int8, device=x.device),
                     self._float(-(-self.F // tc.HGEMM_CKPT8_GROUP), m))

    def forward(self, x):
        """(y, Saved)."""
        saved = self._saved(x, self._rows(x, "x"))
        return self._run(x, saved), saved

    def _run(self, x, s: Saved | None):
        m = self._rows(x, "x")
        h = self._half(m, self.D)
        self._norm(x, h, s and s.mean, s and s.rstd)
        y = self._branch(x, h, s)
        return y if self.plain else self._join(x, y, s, None)[0]

    def _norm(self, x, h, mean, rstd):
        """h = N(x), the norm in front of the block."""
        m, d = x.shape
        if self.layer:
            tc.hgemm_layernorm_forward(x, d, self.gamma, self.beta, self.eps, h, d, mean, rstd, m, d)
            return
        # as the norm behind a branch x, of a stream that counts for nothing
        stats = None if mean is None else self._float(4, m)
        tc.hgemm_residual_norm_forward(x, d, 0.0, x, d, None, self.norm, self.gamma, self.beta, tc.HGEMM_NORM_NONE,
                                       None, None, self.eps, h, d, None, 0, stats, m, d)
        if stats is not None:
            mean.copy_(stats[0])
            rstd.copy_(stats[1])

    def _branch(self, x, h, s: Saved | None):
        """f(h·W1ᵀ + b1)·W2ᵀ + b2, and x added in a plain block."""
        m, d, f = x.shape[0], self.D, self.F
        a, y = self._half(m, f), self._half(m, d)
        tc.hgemm_linear(h, d, self.w1, d, self.b1, self.act, None, 0, a, f, m, f, d,
                        codes=s and s.codes, ldq=f, scales=s and s.scales, lds=max(m, 1))
        tc.hgemm_linear(a, f, self.w2, f, self.b2, tc.HGEMM_ACT_NONE, x if self.plain else None, d, y, d, m, d, f)
        return y

    def _join(self, x, y, s: Saved | None, following):
        """(the residual stream behind this block, the next block's N of it or
        None), y the branch's output (kept in s). following: the next block."""
        m, d = x.shape
        z = self._half(m, d)
        h = None if following is None else self._half(m, d)
        stats = None if s is None else self._float(4, m)
        if s is not None:
            s.y, s.stats = y, stats
        n = following
        tc.hgemm_residual_norm_forward(
            x, d, self.residual_scale, y, d, self.gate, self.post, self.post_gamma, self.post_beta,
            n.norm if n else tc.HGEMM_NORM_NONE, n and n.gamma, n and n.beta, self.eps, z, d, h, d, stats, m, d)
        return z, h

    def _check_saved(self, s: Saved, m):
        """What was saved is read by dy's sizes."""
        d, f = self.D, self.F
        for name, t, shape in (("x", s.x, (m, d)), ("mean", s.mean, (m,)), ("rstd", s.rstd, (m,)),
                               ("codes", s.codes, (m, f)),
                               ("scales", s.scales, (-(-f // tc.HGEMM_CKPT8_GROUP), m)),
                               *((("y", s.y, (m, d)), ("stats", s.stats, (4, m))) if not self.plain else ())):
            if t is None or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"saved {name} must be {shape} and contiguous for this dy, got "
                                 f"{None if t is None else tuple(t.shape)}")

    def backward(self, dy, s: Saved) -> FeedForwardGradients:
        m, d = self._rows(dy, "dy"), self.D
        self._check_saved(s, m)
        grads = FeedForwardGradients(*[None] * 7)
        dx, du = dy, dy
        if not self.plain:
            dx, du = self._join_backward(dy, None, None, None, s, grads, None)
        dh = self._branch_backward(du, None, s, grads)
        # through the norm, the residual branch's gradient added
        if self.layer:
            grads.gamma, grads.beta = self._float(d), self._float(d)
            work = self.torch.empty(tc.hgemm_layernorm_backward_workspace_size(m, d), dtype=self.torch.uint8,
                                    device=dy.device)
            tc.hgemm_layernorm_backward(dh, d, s.x, d, self.gamma, s.mean, s.rstd, dx, d, dh, d, grads.gamma,
                                        grads.beta, work, m, d)
            grads.x = dh
        else:
            grads.x = self._norm_backward(dx, dh, s, grads)
        return grads

    def _work(self, m):
        return self.torch.empty(tc.hgemm_residual_norm_backward_workspace_size(m, self.D), dtype=self.torch.uint8,
                                device=self.w1.device)

    def _norm_backward(self, dx, dh, s: Saved, grads):
        """dx + the gradient through the norm in front of the block; its vectors'."""
        m, d = dh.shape
        grads.gamma, grads.beta = self._float(d), None if self.beta is None else self._float(d)
        stats, out = self._float(4, m), self._half(m, d)
        stats[2].copy_(s.mean)
        stats[3].copy_(s.rstd)
        tc.hgemm_residual_norm_backward(dx, d, dh, d, s.x, d, s.x, d, 1.0, None, tc.HGEMM_NORM_NONE, None, None,
                                        self.norm, self.gamma, stats, out, d, dh, d, None, None, None, grads.gamma,
                                        grads.beta, self._work(m), m, d)
        return out

    def _join_backward(self, dz, dh, z, following, s: Saved, grads, next_grads):
        """(dx along the residual stream, dy of the branch) from dz and, with a
        following block, dh of its N(z)."""
        m, d = dz.shape
        dx, dy = self._half(m, d), self._half(m, d)
        wanted = lambda t: None if t is None else self._float(d)  # noqa: E731
        grads.gate, grads.post_gamma, grads.post_beta = map(wanted, (self.gate, self.post_gamma, self.post_beta))
        n = following
        if n is not None:
            next_grads.gamma, next_grads.beta = wanted(n.gamma), wanted(n.beta)
        tc.hgemm_residual_norm_backward(
            dz, d, dh, d, s.y if z is None else z, d, s.y, d, self.residual_scale, self.gate, self.post,
            self.post_gamma, self.post_beta, n.norm if n else tc.HGEMM_NORM_NONE, n and n.gamma, s.stats, dx, d, dy, d,
            grads.gate, grads.post_gamma, grads.post_beta, n and next_grads.gamma, n and next_grads.beta,
            self._work(m), m, d)
        return dx, dy

    def _branch_backward(self, dy, h, s: Saved, grads):
        """The gradient of h, the norm's output (None: computed again), and those
        of the branch's parameters."""
        m, d, f = dy.shape[0], self.D, self.F
        # through the second product and the activation; a = f(u) comes with it
        du, a = self._half(m, f), self._half(m, f)
        tc.hgemm_linear_dgrad(dy, d, self.w2, f, s.codes, f, s.scales, max(m, 1), self.act, du, f, a, f, m, d, f)
        grads.w2, grads.b2 = self._half(d, f), self._float(d)
        tc.hgemm_linear_wgrad(dy, d, a, f, grads.w2, f, grads.b2, False, m, d, f)
        # through the first product; h = N(x) again
        dh = self._half(m, d)
        if h is None:
            h = self._half(m, d)
            self._norm(s.x, h, None, None)
        grads.w1, grads.b1 = self._half(f, d), self._float(f)
        tc.hgemm_linear_wgrad(du, f, h, d, grads.w1, d, grads.b1, False, m, f, d)
        tc.hgemm_linear_dgrad(du, f, self.w1, d, None, 0, None, 0, tc.HGEMM_ACT_NONE, dh, d, None, 0, m, f, d)
        return dh


class FeedForwardStack:
    """Blocks one behind the other: what lies between two of them, the norm
    behind the first with its gate and residual scale and the norm in front of
    the second, is one pass over the rows each way. Forward a block's input is
    the norm of the stream in 32 bits; backward, for w1's gradient, that of the
    stream as it is kept, rounded to FP16, which is as near as FP16 gradients
    are.

        stack = FeedForwardStack(blocks)
        y = stack(x)
        y, saved = stack.forward(x)
        dx, grads = stack.backward(dy, saved)   # a FeedForwardGradients per block
    """

    def __init__(self, blocks):
        self.blocks = list(blocks)
        if not self.blocks or any((b.D, b.eps) != (self.blocks[0].D, self.blocks[0].eps) for b in self.blocks):
            raise ValueError("a stack needs blocks of one width and one eps")
        if any(b.plain for b in self.blocks[:-1]):
            # a plain block's residual is in its second product's epilogue
            raise ValueError("in a stack every block but the last needs a norm behind it, a gate or a residual scale")

    def __call__(self, x):
        return self._run(x, None)

    def forward(self, x):
        saved = []
        return self._run(x, saved), saved

    def _run(self, x, saved):
        first = self.blocks[0]
        m = first._rows(x, "x")
        h, stats = first._half(m, first.D), None
        for i, b in enumerate(self.blocks):
            s = None if saved is None else b._saved(x, m)
            if i == 0:
                b._norm(x, h, s and s.mean, s and s.rstd)
            elif s is not None:
                s.mean, s.rstd = stats[2], stats[3]  # the pass before has left them
            y = b._branch(x, h, s)
            following = self.blocks[i + 1] if i + 1 < len(self.blocks) else None
            if b.plain:
                x, h = y, None
            else:
                x, h = b._join(x, y, s, following)
            if saved is not None:
                saved.append(s)
                stats = s.stats
        return x

    def backward(self, dy, saved):
        """(dx, the blocks' FeedForwardGradients)."""
        m = self.blocks[0]._rows(dy, "dy")
        if len(saved) != len(self.blocks):
            raise ValueError(f"saved must be of {len(self.blocks)} blocks, got {len(saved)}")
        for b, s in zip(self.blocks, saved):
            b._check_saved(s, m)
        grads = [FeedForwardGradients(*[None] * 7) for _ in self.blocks]
        dx, dh = dy, None
        for i in reversed(range(len(self.blocks))):
            b, s = self.blocks[i], saved[i]
            following = self.blocks[i + 1] if i + 1 < len(self.blocks) else None
            du = dx
            if not b.plain:
                # (x of the block behind is the stream between the two)
                dx, du = b._join_backward(dx, dh, saved[i + 1].x if following else None, following, s, grads[i],
                                          grads[i + 1] if following else None)
            dh = b._branch_backward(du, None, s, grads[i])
        first = self.blocks[0]
        grads[0].x = first._norm_backward(dx, dh, saved[0], grads[0])
        return grads[0].x, grads


class ExpertFeedForward:
    """A mixture-of-experts layer of the block's kind, for tokens: each row goes
    through the k experts of E that the router chooses for it.

        layer = ExpertFeedForward(router, w1, w2, k=2, act="silu", gated=True)
        y = layer(h, residual=x)

    router E×D, w1 E×F×D (gated: E×2F×D, the gates first), w2 E×D×F, b1 E×F (2F)
    and b2 E×D or None; CUDA FP16, contiguous. Rows are taken 64 at a time."""

    def __init__(self, router, w1, w2, b1=None, b2=None, k: int = 2, act: str = "silu", gated: bool = True,
                 normalize: bool = True):
        import torch
        self.torch = torch
        self.E, self.D = router.shape
        self.F = w2.shape[2]
        up = 2 * self.F if gated else self.F
        for name, t, shape in (("router", router, (self.E, self.D)), ("w1", w1, (self.E, up, self.D)),
                               ("w2", w2, (self.E, self.D, self.F)), ("b1", b1, (self.E, up)),
                               ("b2", b2, (self.E, self.D))):
            if t is None and name in ("b1", "b2"):
                continue
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if not 1 <= k <= min(self.E, tc.HGEMM_EXPERTS_MAX_CHOICES):
            raise ValueError(f"k must be 1 to {min(self.E, tc.HGEMM_EXPERTS_MAX_CHOICES)}, got {k}")
        self.router, self.w1, self.w2, self.b1, self.b2 = router, w1, w2, b1, b2
        self.k, self.act, self.gated, self.normalize = k, ACTIVATIONS[act], gated, normalize

    def __call__(self, x, residual=None, choices: bool = False):
        """Y (and with choices the experts chosen, M×k, and their shares)."""
        torch, d, k = self.torch, self.D, self.k
        for name, t in (("x", x), ("residual", residual)):
            if t is not None and (t.dim() != 2 or t.shape[1] != d or not t.is_contiguous()
                                  or t.shape[0] != x.shape[0]):
                raise ValueError(f"{name} must be a contiguous M×{d} matrix")
        m = x.shape[0]
        y = torch.empty_like(x)
        chosen = torch.empty((m, k), dtype=torch.int32, device=x.device)
        share = torch.empty((m, k), dtype=torch.float32, device=x.device)
        most = tc.HGEMM_EXPERTS_MAX_TOKENS
        work = torch.empty(tc.hgemm_experts_workspace_size(min(m, most), d, self.F, self.E, k), dtype=torch.uint8,
                           device=x.device)
        for i in range(0, m, most):
            rows = slice(i, min(i + most, m))
            tc.hgemm_experts(x[rows], d, self.router, d, self.w1, d, self.b1, self.w2, self.F, self.b2, self.act,
                             self.gated, k, self.normalize, None if residual is None else residual[rows], d, y[rows], d,
                             chosen[rows], share[rows], work, rows.stop - i, d, self.F, self.E)
        return (y, chosen, share) if choices else y


class AdamW:
    """AdamW over FP16 parameters by name: FP32 copies (master) and FP32 or 8-bit
    states, all stepped by one launch.

        optimizer = AdamW(block.parameters(), lr=1e-3, bits=8)
        optimizer.step(block.backward(dy, saved).named())

    weight_decay goes to parameters of two dimensions alone, unless `decay`
    names which. 8-bit states are rounded at random, by the values' indexes and
    the step's number, so that they follow their gradients over many steps and
    equal runs are equal.

    `tensors` holds a dict of what hgemm_adamw_tensors takes for each of `names`,
    without the gradient. Its states, master copies and weight_decay may be
    replaced or given other values between steps (a checkpoint, a schedule), and
    `steps` counts the steps so far. With master copies a step reads those and
    overwrites the weights: who sets weights sets them too. Under a captured
    graph a step's learning rate, number and scale come from `dynamic`."""

    def __init__(self, parameters, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.01, bits: int = 32, master: bool = True, decay=None):
        import torch
        if bits not in (8, 32):
            raise ValueError(f"bits must be 8 or 32, got {bits}")
        self.lr, self.beta1, self.beta2, self.eps, self.steps = lr, beta1, beta2, eps, 0
        self.names, self.tensors, self.plan, self._held = list(parameters), [], None, None
        for name in self.names:
            p = parameters[name]
            n = p.numel()

            def zeros(dtype, size=n, like=p):
                return torch.zeros(size, dtype=dtype, device=like.device)

            t = {"weight": p, "master": p.float() if master else None,
                 "weight_decay": weight_decay if (p.dim() > 1 if decay is None else name in decay) else 0.0}
            if bits == 8:
                groups = -(-n // tc.HGEMM_CKPT8_GROUP)
                t.update(m=zeros(torch.int8), v=zeros(torch.uint8), m_scales=zeros(torch.float32, groups),
                         v_scales=zeros(torch.float32, groups))
            else:
                t.update(m=zeros(torch.float32), v=zeros(torch.float32))
            self.tensors.append(t)

    def step(self, gradients, grad_scale: float = 1.0, dynamic=None, stream=None) -> None:
        """One step with the gradients of these names (float16 or float32).
        dynamic: see hgemm_adamw."""
        grads = [gradients[name] for name in self.names]
        if self.plan is not None and self._unchanged():
            self.plan.set_gradients(grads)
        else:
            self.plan = tc.hgemm_adamw_tensors({**t, "grad": g} for t, g in zip(self.tensors, grads))
            held, decays = self._entries()
            self._held = held, self._addresses(held), decays
        tc.hgemm_adamw_rounded(self.plan, self.lr, self.beta1, self.beta2, self.eps, self.steps + 1, grad_scale,
                               tc.HGEMM_ROUND_RANDOM, dynamic, stream)
        self.steps += 1  # (a refused step is none)

    def _entries(self):
        """What a table holds of `tensors`: the tensors, in order, and the decays."""
        return ([t.get(n) for t in self.tensors for n in ("weight", "master", "m", "v", "m_scales", "v_scales")],
                [t.get("weight_decay", 0.0) for t in self.tensors])

    @staticmethod
    def _addresses(held):
        return [None if x is None else x.data_ptr() for x in held]

    def _unchanged(self) -> bool:
        """Whether the table says what `tensors` does: the same tensors, where
        they were, and the same decays."""
        held, at, decays = self._held
        now, now_decays = self._entries()
        return (now_decays == decays and len(now) == len(held) and all(map(operator.is_, now, held))
                and self._addresses(held) == at)


def main() -> None:
    import torch
    m, d, f = 4096, 2048, 8192
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).half()

    block = FeedForward(1 + normal(d, scale=0.1), normal(d, scale=0.1), normal(f, d, scale=d ** -0.5),
                        normal(f, scale=0.1), normal(d, f, scale=f ** -0.5), normal(d, scale=0.1))
    x, dy = normal(m, d), normal(m, d, scale=0.05)

    def timed(what, call, count=20):
        for _ in range(3):
            call()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record()
        for _ in range(count):
            call()
        end.record()
        torch.cuda.synchronize()
        print(f"{what}: {start.elapsed_time(end) / count * 1e3:.1f} us")

    def step():
        y, saved = block.forward(x)
        return block.backward(dy, saved)

    timed(f"training step, {m} tokens, {d} -> {f} -> {d}", step)
    grads = step().named()
    for bits in (32, 8):
        optimizer = AdamW(block.parameters(), lr=1e-5, bits=bits)
        timed(f"AdamW, states in {bits} bits", lambda: optimizer.step(grads))
    sandwich = [FeedForward(**block.parameters(), post="rms", post_gamma=1 + normal(d, scale=0.1),
                            gate=normal(d, scale=0.1)) for _ in range(2)]
    stack = FeedForwardStack(sandwich)

    def stack_step():
        y, saved = stack.forward(x)
        return stack.backward(dy, saved)

    timed("two blocks with a norm and a gate behind each", stack_step)
    one = x[:1].contiguous()
    timed("one token", lambda: block(one))
    experts = ExpertFeedForward(normal(8, d, scale=2 * d ** -0.5), normal(8, 2 * f, d, scale=d ** -0.5),
                                normal(8, d, f, scale=f ** -0.5))
    timed("one token through two of eight experts", lambda: experts(one, residual=one))
    if tc.hgemm_device_status() != tc.HGEMM_OK:
        raise RuntimeError("a kernel wait timed out")


if __name__ == "__main__":
    main()
