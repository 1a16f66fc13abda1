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
needs their derivative anyway. ``python -m tensor_core_dense_fp16_gb300.feedforward``
runs a training step and a token.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Any

import tensor_core_dense_fp16_gb300 as tc

ACTIVATIONS = {"none": tc.HGEMM_ACT_NONE, "relu": tc.HGEMM_ACT_RELU, "gelu": tc.HGEMM_ACT_GELU,
               "silu": tc.HGEMM_ACT_SILU, "gelu_erf": tc.HGEMM_ACT_GELU_ERF}


@dataclass
class Saved:
    """What the backward pass needs of a forward pass."""
    x: Any
    mean: Any
    rstd: Any
    codes: Any   # M×F signed bytes
    scales: Any  # ⌈F/64⌉×M


@dataclass
class FeedForwardGradients:
    x: Any
    gamma: Any
    beta: Any
    w1: Any
    b1: Any
    w2: Any
    b2: Any


class FeedForward:
    def __init__(self, gamma, beta, w1, b1, w2, b2, act: str = "gelu", eps: float = 1e-5):
        import torch
        self.torch = torch
        self.F, self.D = w1.shape
        for name, t, shape in (("gamma", gamma, (self.D,)), ("beta", beta, (self.D,)), ("w1", w1, (self.F, self.D)),
                               ("b1", b1, (self.F,)), ("w2", w2, (self.D, self.F)), ("b2", b2, (self.D,))):
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.gamma, self.beta, self.w1, self.b1, self.w2, self.b2 = gamma, beta, w1, b1, w2, b2
        self.act, self.eps = ACTIVATIONS[act], eps

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

    def forward(self, x):
        """(y, Saved)."""
        m = self._rows(x, "x")
        saved = Saved(x, self._float(m), self._float(m),
                      self.torch.empty((m, self.F), dtype=self.torch.int8, device=x.device),
                      self._float(-(-self.F // tc.HGEMM_CKPT8_GROUP), m))
        return self._run(x, saved), saved

    def _run(self, x, s: Saved | None):
        m, d, f = self._rows(x, "x"), self.D, self.F
        h, a, y = self._half(m, d), self._half(m, f), self._half(m, d)
        tc.hgemm_layernorm_forward(x, d, self.gamma, self.beta, self.eps, h, d, s and s.mean, s and s.rstd, m, d)
        tc.hgemm_linear(h, d, self.w1, d, self.b1, self.act, None, 0, a, f, m, f, d,
                        codes=s and s.codes, ldq=f, scales=s and s.scales, lds=max(m, 1))
        tc.hgemm_linear(a, f, self.w2, f, self.b2, tc.HGEMM_ACT_NONE, x, d, y, d, m, d, f)
        return y

    def backward(self, dy, s: Saved) -> FeedForwardGradients:
        m, d, f = self._rows(dy, "dy"), self.D, self.F
        # what was saved is read by dy's sizes
        for name, t, shape in (("x", s.x, (m, d)), ("mean", s.mean, (m,)), ("rstd", s.rstd, (m,)),
                               ("codes", s.codes, (m, f)),
                               ("scales", s.scales, (-(-f // tc.HGEMM_CKPT8_GROUP), m))):
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"saved {name} must be {shape} and contiguous for this dy, got {tuple(t.shape)}")
        # through the second product and the activation; a = f(u) comes with it
        du, a = self._half(m, f), self._half(m, f)
        tc.hgemm_linear_dgrad(dy, d, self.w2, f, s.codes, f, s.scales, max(m, 1), self.act, du, f, a, f, m, d, f)
        dw2, db2 = self._half(d, f), self._float(d)
        tc.hgemm_linear_wgrad(dy, d, a, f, dw2, f, db2, False, m, d, f)
        # through the first product; h = LN(x) again
        h, dh = self._half(m, d), self._half(m, d)
        tc.hgemm_layernorm_forward(s.x, d, self.gamma, self.beta, self.eps, h, d, None, None, m, d)
        dw1, db1 = self._half(f, d), self._float(f)
        tc.hgemm_linear_wgrad(du, f, h, d, dw1, d, db1, False, m, f, d)
        tc.hgemm_linear_dgrad(du, f, self.w1, d, None, 0, None, 0, tc.HGEMM_ACT_NONE, dh, d, None, 0, m, f, d)
        # through the norm, the residual branch's gradient added
        dgamma, dbeta = self._float(d), self._float(d)
        work = self.torch.empty(tc.hgemm_layernorm_backward_workspace_size(m, d), dtype=self.torch.uint8,
                                device=dy.device)
        tc.hgemm_layernorm_backward(dh, d, s.x, d, self.gamma, s.mean, s.rstd, dy, d, dh, d, dgamma, dbeta, work, m, d)
        return FeedForwardGradients(dh, dgamma, dbeta, dw1, db1, dw2, db2)


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
    one = x[:1].contiguous()
    timed("one token", lambda: block(one))
    if tc.hgemm_device_status() != tc.HGEMM_OK:
        raise RuntimeError("a kernel wait timed out")


if __name__ == "__main__":
    main()
