"""The operators of a transformer's feed-forward block, measured one by one.

The block is h = LN(x); a = act(h·W1ᵀ + b1); y = a·W2ᵀ + b2 + x, trained with
the pre-activations kept in 8 bits and served token by token. Its operators:

  linear      Y = act(X·Wᵀ + b) + R, optionally keeping U = X·Wᵀ + b in 8 bits
  dgrad       dU = (dY·W) ⊙ act'(Û) and H = act(Û), Û read back from 8 bits
  wgrad       dW = dYᵀ·X and db = Σ_rows dY
  layernorm   forward (y, mean, 1/σ), and backward (dx with the residual
              branch's gradient added, dγ, dβ)
  ckpt8       keeping a matrix in 8 bits and reading it back

The 8-bit form: in each row, every 64 consecutive columns share a scale
s = max|u| / 127, and a value is kept as the whole number round(u·127/max|u|).

``own`` False computes each operator in its plain form with elementary torch
operations in 32 bits; ``own`` True calls the library.
"""

import math

import torch

own = False

GROUP = 64
ACTS = ("none", "relu", "gelu", "silu", "gelu_erf")  # in the order of HGEMM_ACT_*
EPS = 1e-5


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one generated token through the block's first product: the weights' bytes are all there is
        {"name": "linear_token", "op": "linear", "M": 1, "N": 8192, "K": 2048, "act": "gelu", "bias": True,
         "residual": False, "keep": False},
        # a small batch of generated tokens through the second product, added to the residual stream
        {"name": "linear_batch", "op": "linear", "M": 24, "N": 2048, "K": 8192, "act": "none", "bias": True,
         "residual": True, "keep": False},
        # a short prompt of odd length and ragged features
        {"name": "linear_ragged", "op": "linear", "M": 1000, "N": 1000, "K": 1000, "act": "silu", "bias": True,
         "residual": True, "keep": False},
        # a training step's first product, its pre-activations kept in 8 bits for the backward pass
        {"name": "linear_train", "op": "linear", "M": 8192, "N": 8192, "K": 2048, "act": "gelu", "bias": True,
         "residual": False, "keep": True},
        # backward through the second product and the activation: a small ragged step
        {"name": "dgrad_ragged", "op": "dgrad", "M": 1000, "N": 1000, "K": 1000, "act": "silu", "hidden": True},
        # the same at a training step's size
        {"name": "dgrad_train", "op": "dgrad", "M": 8192, "N": 2048, "K": 8192, "act": "gelu", "hidden": True},
        # gradients of a weight and its bias: a small ragged step
        {"name": "wgrad_ragged", "op": "wgrad", "M": 1000, "N": 1000, "K": 1000, "bias": True},
        # the same at a training step's size
        {"name": "wgrad_train", "op": "wgrad", "M": 8192, "N": 8192, "K": 2048, "bias": True},
        # the norm of one generated token: latency
        {"name": "layernorm_token", "op": "layernorm", "M": 1, "D": 4096, "dir": "forward", "residual": False},
        # the norm's backward pass in training: two inputs, the residual branch and one output streamed
        {"name": "layernorm_train", "op": "layernorm", "M": 16384, "D": 8192, "dir": "backward", "residual": True},
        # keeping a ragged activation
        {"name": "ckpt8_ragged", "op": "ckpt8", "M": 257, "N": 1000},
        # keeping a training step's activation
        {"name": "ckpt8_train", "op": "ckpt8", "M": 16384, "N": 8192},
    ]


MOST_MACS = 8192 * 8192 * 2048  # of a product
MOST_ELEMENTS = 16384 * 8192    # of a streamed matrix


def draw(rng):
    """One more case: sizes spread over their logarithm, feature counts mostly multiples of 8, some odd."""
    def size(lo, hi, step=1):
        n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
        n = max(step, n // step * step) if step > 1 else n
        return n + step if n == 3072 else n

    def features(hi):
        return size(64, hi, 8) if rng.random() < 0.8 else size(64, hi) | 1

    op = rng.choice(("linear", "linear", "dgrad", "wgrad", "layernorm", "ckpt8"))
    while True:
        if op in ("linear", "dgrad", "wgrad"):
            c = {"op": op, "M": size(1, 8192) if op == "linear" else size(16, 8192), "N": features(8192),
                 "K": features(8192)}
            if c["M"] * c["N"] * c["K"] > MOST_MACS:
                continue
            if op == "linear":
                c.update(act=rng.choice(ACTS), bias=rng.random() < 0.8, residual=rng.random() < 0.5,
                         keep=rng.random() < 0.4)
            elif op == "dgrad":
                c.update(act=rng.choice(ACTS[1:]), hidden=rng.random() < 0.5)
            else:
                c.update(bias=rng.random() < 0.8)
            return c
        if op == "layernorm":
            c = {"op": op, "M": size(1, 16384), "D": features(16384), "dir": rng.choice(("forward", "backward")),
                 "residual": rng.random() < 0.5}
            c["residual"] = c["residual"] and c["dir"] == "backward"
            if c["M"] * c["D"] <= MOST_ELEMENTS:
                return c
            continue
        c = {"op": op, "M": size(1, 16384), "N": features(16384)}
        if c["M"] * c["N"] <= MOST_ELEMENTS:
            return c


# -------------------------------------------------------------------- the inputs

def _normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).half()


def _activations(g, m, n):
    """What a norm's output looks like: unit variance, a few columns much larger than the rest."""
    x = torch.randn((m, n), generator=g, device="cuda", dtype=torch.float32)
    col = torch.rand((n,), generator=g, device="cuda")
    return (x * torch.where(col > 0.99, 6.0, 1.0)).half()


def _kept(g, m, n):
    """A matrix kept in 8 bits, as whole numbers and scales: pre-activations of unit variance."""
    groups = -(-n // GROUP)
    codes = torch.empty((m, n), device="cuda", dtype=torch.int8)
    scales = torch.empty((groups, m), device="cuda", dtype=torch.float32)
    _keep(torch.randn((m, n), generator=g, device="cuda", dtype=torch.float32), codes, scales)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]
    s = {"case": case, "act": ACTS.index(c.get("act", "none"))}
    f16 = {"device": "cuda", "dtype": torch.float16}
    f32 = {"device": "cuda", "dtype": torch.float32}
    if op == "linear":
        m, n, k = c["M"], c["N"], c["K"]
        s["x"] = _activations(g, m, k)
        s["w"] = _normal(g, (n, k), 1 / math.sqrt(k))
        s["b"] = _normal(g, (n,), 0.1) if c["bias"] else None
        s["r"] = _normal(g, (m, n), 2.0) if c["residual"] else None
        s["y"] = torch.empty((m, n), **f16)
        if c["keep"]:
            s["codes"] = torch.empty((m, n), device="cuda", dtype=torch.int8)
            s["scales"] = torch.empty((-(-n // GROUP), m), **f32)
            s["u"] = torch.empty((m, n), **f16)
    elif op == "dgrad":
        m, n, k = c["M"], c["N"], c["K"]
        s["dy"] = _normal(g, (m, n), 0.05)
        s["w"] = _normal(g, (n, k), 1 / math.sqrt(n))
        s["codes"], s["scales"] = _kept(g, m, k)
        s["du"] = torch.empty((m, k), **f16)
        s["h"] = torch.empty((m, k), **f16) if c["hidden"] else None
    elif op == "wgrad":
        m, n, k = c["M"], c["N"], c["K"]
        s["dy"] = _normal(g, (m, n), 0.05)
        s["x"] = _activations(g, m, k)
        s["dw"] = torch.empty((n, k), **f16)
        s["db"] = torch.empty((n,), **f32) if c["bias"] else None
    elif op == "layernorm":
        m, d = c["M"], c["D"]
        s["x"] = (_activations(g, m, d).float() * 1.5 + 0.25).half()
        s["gamma"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")).half()
        s["beta"] = _normal(g, (d,), 0.1)
        s["mean"], s["rstd"] = torch.empty((m,), **f32), torch.empty((m,), **f32)
        if c["dir"] == "forward":
            s["y"] = torch.empty((m, d), **f16)
        else:
            x = s["x"].float()
            var, mu = torch.var_mean(x, dim=1, correction=0)
            s["mean"].copy_(mu)
            s["rstd"].copy_(torch.rsqrt(var + EPS))
            s["dy"] = _normal(g, (m, d), 0.05)
            s["r"] = _normal(g, (m, d), 0.05) if c["residual"] else None
            s["dx"] = torch.empty((m, d), **f16)
            s["dgamma"], s["dbeta"] = torch.empty((d,), **f32), torch.empty((d,), **f32)
            # the backward pass's scratch: two rows of partial sums for each of up to 1024 groups of rows
            s["work"] = torch.empty((1024 * 2 * (d + 32),), **f32)
    else:
        m, n = c["M"], c["N"]
        s["x"] = _activations(g, m, n)
        s["codes"] = torch.empty((m, n), device="cuda", dtype=torch.int8)
        s["scales"] = torch.empty((-(-n // GROUP), m), **f32)
        s["u"] = torch.empty((m, n), **f16)
    return s


# --------------------------------------------------------------- the plain forms

def _act(u, act):
    if act == 1:
        return torch.where(u < 0, torch.zeros_like(u), u)
    if act == 2:
        return 0.5 * u * (1 + torch.tanh(0.7978845608028654 * (u + 0.044715 * u * u * u)))
    if act == 3:
        return u / (1 + torch.exp(-u))
    if act == 4:
        return 0.5 * u * (1 + torch.erf(u * 0.7071067811865476))
    return u


def _act_gradient(u, act):
    if act == 1:
        return (u > 0).float()
    if act == 2:
        t = torch.tanh(0.7978845608028654 * (u + 0.044715 * u * u * u))
        return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * u * u)
    if act == 3:
        p = 1 / (1 + torch.exp(-u))
        return p * (1 + u * (1 - p))
    if act == 4:
        return 0.5 * (1 + torch.erf(u * 0.7071067811865476)) + u * torch.exp(-0.5 * u * u) * 0.3989422804014327
    return torch.ones_like(u)


def _keep(u, codes, scales):
    """u (32 bits) into whole numbers and scales."""
    m, n = u.shape
    groups = -(-n // GROUP)
    if n % GROUP:
        u = torch.cat([u, u.new_zeros((m, groups * GROUP - n))], dim=1)
    v = u.view(m, groups, GROUP)
    top = v.abs().amax(dim=2, keepdim=True)
    q = torch.where(top > 0, torch.round(v * (127.0 / top)), torch.zeros_like(v))
    codes.copy_(q.view(m, groups * GROUP)[:, :n])
    scales.copy_((top[:, :, 0] / 127.0).t())


def _kept_values(codes, scales):
    n = codes.shape[1]
    return codes.float() * scales.t().repeat_interleave(GROUP, dim=1)[:, :n]


def _plain(s):
    c, act = s["case"], s["act"]
    op = c["op"]
    if op == "linear":
        u = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            u = u + s["b"].float()
        y = _act(u, act)
        if s["r"] is not None:
            y = y + s["r"].float()
        if not c["keep"]:
            return {"y": y.half()}
        _keep(u, s["codes"], s["scales"])
        return {"y": y.half(), "u": _kept_values(s["codes"], s["scales"]).half()}
    if op == "dgrad":
        u = _kept_values(s["codes"], s["scales"])
        du = (s["dy"].float() @ s["w"].float()) * _act_gradient(u, act)
        out = {"du": du.half()}
        if c["hidden"]:
            out["h"] = _act(u, act).half()
        return out
    if op == "wgrad":
        dy = s["dy"].float()
        out = {"dw": (dy.t() @ s["x"].float()).half()}
        if s["db"] is not None:
            out["db"] = dy.sum(dim=0)
        return out
    if op == "layernorm":
        x, gamma = s["x"].float(), s["gamma"].float()
        if c["dir"] == "forward":
            mu = x.mean(dim=1, keepdim=True)
            rstd = 1 / torch.sqrt((x - mu).square().mean(dim=1, keepdim=True) + EPS)
            y = (x - mu) * rstd * gamma + s["beta"].float()
            return {"y": y.half(), "mean": mu[:, 0], "rstd": rstd[:, 0]}
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        gy = dy * gamma
        dx = rstd * (gy - gy.mean(dim=1, keepdim=True) - xh * (gy * xh).mean(dim=1, keepdim=True))
        if s["r"] is not None:
            dx = dx + s["r"].float()
        return {"dx": dx.half(), "dgamma": (dy * xh).sum(dim=0), "dbeta": dy.sum(dim=0)}
    _keep(s["x"].float(), s["codes"], s["scales"])
    return {"u": _kept_values(s["codes"], s["scales"]).half()}


# ------------------------------------------------------------ the library's calls

def _library(s):
    import tensor_core_dense_fp16_gb300 as tc
    c, act = s["case"], s["act"]
    op, m = c["op"], c["M"]
    if op == "linear":
        n, k = c["N"], c["K"]
        if not c["keep"]:
            tc.hgemm_linear(s["x"], k, s["w"], k, s["b"], act, s["r"], n, s["y"], n, m, n, k)
            return {"y": s["y"]}
        tc.hgemm_linear(s["x"], k, s["w"], k, s["b"], act, s["r"], n, s["y"], n, m, n, k,
                        codes=s["codes"], ldq=n, scales=s["scales"], lds=m)
        tc.hgemm_ckpt8_load(s["codes"], n, s["scales"], m, tc.HGEMM_ACT_NONE, s["u"], n, m, n)
        return {"y": s["y"], "u": s["u"]}
    if op == "dgrad":
        n, k = c["N"], c["K"]
        tc.hgemm_linear_dgrad(s["dy"], n, s["w"], k, s["codes"], k, s["scales"], m, act, s["du"], k, s["h"], k,
                              m, n, k)
        return {"du": s["du"], "h": s["h"]} if c["hidden"] else {"du": s["du"]}
    if op == "wgrad":
        n, k = c["N"], c["K"]
        tc.hgemm_linear_wgrad(s["dy"], n, s["x"], k, s["dw"], k, s["db"], False, m, n, k)
        return {"dw": s["dw"], "db": s["db"]} if s["db"] is not None else {"dw": s["dw"]}
    if op == "layernorm":
        d = c["D"]
        if c["dir"] == "forward":
            tc.hgemm_layernorm_forward(s["x"], d, s["gamma"], s["beta"], EPS, s["y"], d, s["mean"], s["rstd"], m, d)
            return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        tc.hgemm_layernorm_backward(s["dy"], d, s["x"], d, s["gamma"], s["mean"], s["rstd"], s["r"], d, s["dx"], d,
                                    s["dgamma"], s["dbeta"], s["work"], m, d)
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    n = c["N"]
    tc.hgemm_ckpt8_save(s["x"], n, s["codes"], n, s["scales"], m, m, n)
    tc.hgemm_ckpt8_load(s["codes"], n, s["scales"], m, tc.HGEMM_ACT_NONE, s["u"], n, m, n)
    return {"u": s["u"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------- the work of a pass

def work(case):
    c, op, m = case, case["op"], case["M"]
    if op in ("linear", "dgrad", "wgrad"):
        n, k = c["N"], c["K"]
        flops = 2 * m * n * k
        if op == "linear":
            by = 2 * (m * k + n * k + m * n) + (2 * n if c["bias"] else 0) + (2 * m * n if c["residual"] else 0)
            if c["keep"]:  # 8-bit values and scales written, and the values they stand for
                by += m * n + 4 * m * -(-n // GROUP) + 2 * m * n
        elif op == "dgrad":
            by = 2 * (m * n + n * k + m * k) + m * k + 4 * m * -(-k // GROUP) + (2 * m * k if c["hidden"] else 0)
        else:
            by = 2 * (m * n + m * k + n * k) + (4 * n if c["bias"] else 0)
            flops += m * n if c["bias"] else 0
        return {"bytes": by, "flops": flops}
    if op == "layernorm":
        d = c["D"]
        if c["dir"] == "forward":
            return {"bytes": 4 * m * d + 4 * d + 8 * m, "flops": 8 * m * d}
        return {"bytes": (6 + (2 if c["residual"] else 0)) * m * d + 8 * m + 10 * d, "flops": 14 * m * d}
    n = c["N"]
    return {"bytes": 4 * m * n + 2 * (m * n + 4 * m * -(-n // GROUP)), "flops": 4 * m * n}


# ----------------------------------------------------------------- in 64 bits

def _act64(u, name):
    """The activation's definition; its derivative is taken of this."""
    if name == "relu":
        return torch.relu(u)
    if name == "gelu":  # u·σ(2z), z the tanh's argument
        return u * torch.sigmoid(math.sqrt(8 / math.pi) * (u + 0.044715 * u.pow(3)))
    if name == "silu":
        return u * torch.sigmoid(u)
    if name == "gelu_erf":  # u·Φ(u)
        return u * 0.5 * torch.erfc(-u / math.sqrt(2))
    return u * 1


def _spread64(codes, scales):
    u = torch.empty(codes.shape, device=codes.device, dtype=torch.float64)
    for g in range(scales.shape[0]):
        cols = slice(g * GROUP, (g + 1) * GROUP)
        u[:, cols] = codes[:, cols].double() * scales[g].double()[:, None]
    return u


def exact(case, seed):
    """Each output before its rounding (to 16 or to 8 bits)."""
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "linear":
        u = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
        if s["b"] is not None:
            u += s["b"].double()[None, :]
        y = _act64(u, c["act"])
        if s["r"] is not None:
            y += s["r"].double()
        return {"y": y, "u": u} if c["keep"] else {"y": y}
    if op == "dgrad":
        u = _spread64(s["codes"], s["scales"]).requires_grad_()
        h = _act64(u, c["act"])
        du, = torch.autograd.grad(h, u, torch.einsum("mn,nk->mk", s["dy"].double(), s["w"].double()))
        return {"du": du, "h": h.detach()} if c["hidden"] else {"du": du}
    if op == "wgrad":
        out = {"dw": torch.einsum("mn,mk->nk", s["dy"].double(), s["x"].double())}
        if s["db"] is not None:
            out["db"] = torch.einsum("mn->n", s["dy"].double())
        return out
    if op == "layernorm":
        x = s["x"].double()
        gamma, beta = s["gamma"].double(), s["beta"].double()
        if c["dir"] == "forward":
            var, mu = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            rstd = (var + EPS).rsqrt()
            return {"y": torch.addcmul(beta, (x - mu) * rstd, gamma), "mean": mu[:, 0], "rstd": rstd[:, 0]}
        # by projection: the part of γ·dy along 1 and along the normalised row is taken out
        xh = torch.addcmul(-(s["mean"].double() * s["rstd"].double())[:, None], x, s["rstd"].double()[:, None])
        dy = s["dy"].double()
        dgamma, dbeta = torch.einsum("md,md->d", dy, xh), torch.einsum("md->d", dy)
        gy = dy * gamma
        d = x.shape[1]
        along = torch.einsum("md,md->m", gy, xh) / d
        gy -= (torch.einsum("md->m", gy) / d)[:, None]
        gy -= along[:, None] * xh
        gy *= s["rstd"].double()[:, None]
        if s["r"] is not None:
            gy += s["r"].double()
        return {"dx": gy, "dgamma": dgamma, "dbeta": dbeta}
    return {"u": s["x"].double()}
