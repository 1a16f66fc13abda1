"""The operators around a transformer's feed-forward block, measured one by one.

  residual_norm   z = alpha·x + gate ⊙ N(y), h = N'(z): the norm behind a block
                  with the block's gate and the residual scale, and the norm in
                  front of the next one; forward, and backward (dx, dy and the
                  gradients of the gate and of both norms' vectors)
  adamw           one AdamW step over many tensors at once, the states in 32 or
                  in 8 bits
  experts         a mixture-of-experts feed-forward layer for few tokens:
                  router, the chosen experts' two products, their weighted sum

N(v) = (v − μ)·ρ·gamma + beta over rows: a layer norm, or with μ = 0 an RMS norm.

The 8-bit states: every 64 consecutive values of a tensor share two scales.
m: s = max|m| / 127, kept as round(m·(127/max|m|)). v: s = max v, and v/s is
kept as an unsigned float of 5 exponent and 3 fraction bits, of which 255
stands for 1, 1 for the least and 0 for zero.

``own`` False computes each operator in its plain form with elementary torch
operations in 32 bits; ``own`` True calls the library.
"""

import math

import torch

own = False

GROUP = 64
NORMS = ("none", "layer", "rms")                     # in the order of HGEMM_NORM_*
ACTS = ("none", "relu", "gelu", "silu", "gelu_erf")  # in the order of HGEMM_ACT_*
EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.01, 100


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # behind a block, one generated token: latency
        {"name": "norm_token", "op": "residual_norm", "M": 1, "D": 4096, "dir": "forward", "post": "rms", "pre": "rms",
         "gate": False, "alpha": 1.0},
        # a training step's rows, both norms and a gate
        {"name": "norm_train", "op": "residual_norm", "M": 16384, "D": 4096, "dir": "forward", "post": "rms",
         "pre": "rms", "gate": True, "alpha": 1.0},
        # back through a small ragged step
        {"name": "norm_back_ragged", "op": "residual_norm", "M": 1000, "D": 1000, "dir": "backward", "post": "layer",
         "pre": "layer", "gate": True, "alpha": 0.75},
        # the same at a training step's size: four matrices read, two written
        {"name": "norm_back_train", "op": "residual_norm", "M": 16384, "D": 8192, "dir": "backward", "post": "rms",
         "pre": "rms", "gate": True, "alpha": 1.0},
        # the vectors of a few blocks: latency
        {"name": "adamw_vectors", "op": "adamw", "bits": 32, "weights": 0, "rows": 1, "cols": 2048, "vectors": 6,
         "master": True},
        # a feed-forward block's six tensors, states and a copy of the weights in 32 bits
        {"name": "adamw_block", "op": "adamw", "bits": 32, "weights": 2, "rows": 8192, "cols": 2048, "vectors": 4,
         "master": True},
        # many small ragged tensors with states in 8 bits
        {"name": "adamw_8bit_ragged", "op": "adamw", "bits": 8, "weights": 24, "rows": 257, "cols": 1000, "vectors": 48,
         "master": False},
        # a stack of blocks with states in 8 bits
        {"name": "adamw_8bit_stack", "op": "adamw", "bits": 8, "weights": 24, "rows": 4096, "cols": 1024, "vectors": 96,
         "master": False},
        # one generated token through two of eight large experts: the weights' bytes are all there is
        {"name": "experts_token", "op": "experts", "M": 1, "D": 2048, "F": 8192, "E": 8, "k": 2, "act": "silu",
         "gated": True, "bias": False, "residual": False, "normalize": True},
        # a few tokens through ragged experts of the block's own kind: biases, no gate
        {"name": "experts_ragged", "op": "experts", "M": 7, "D": 1000, "F": 1000, "E": 10, "k": 3, "act": "gelu",
         "gated": False, "bias": True, "residual": True, "normalize": True},
        # a batch of generated tokens through many small experts
        {"name": "experts_batch", "op": "experts", "M": 24, "D": 2048, "F": 1024, "E": 64, "k": 8, "act": "silu",
         "gated": True, "bias": False, "residual": True, "normalize": True},
        # the most tokens a call takes
        {"name": "experts_most", "op": "experts", "M": 64, "D": 4096, "F": 1024, "E": 64, "k": 4, "act": "silu",
         "gated": True, "bias": False, "residual": True, "normalize": False},
    ]


MOST_ROWS_VALUES = 16384 * 8192             # of a matrix of rows
MOST_VALUES = 24 * 4096 * 1024 + 96 * 1024  # of an optimizer step
MOST_EXPERTS_VALUES = 64 * 3 * 4096 * 1024  # of a layer's experts


def draw(rng):
    """One more case: sizes spread over their logarithm, feature counts mostly multiples of 8, some odd."""
    def size(lo, hi, step=1):
        n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
        return max(step, n // step * step) if step > 1 else n

    def features(hi):
        return size(64, hi, 8) if rng.random() < 0.8 else size(64, hi) | 1

    op = rng.choice(("residual_norm", "adamw", "experts"))
    while True:
        if op == "residual_norm":
            c = {"op": op, "M": size(1, 16384), "D": features(8192), "dir": rng.choice(("forward", "backward")),
                 "post": rng.choice(NORMS), "pre": rng.choice(NORMS), "gate": rng.random() < 0.6,
                 "alpha": rng.choice((1.0, 1.0, 0.75, 2.0))}
            if c["M"] * c["D"] <= MOST_ROWS_VALUES:
                return c
        elif op == "adamw":
            c = {"op": op, "bits": rng.choice((8, 32)), "weights": rng.randint(0, 48), "rows": size(1, 8192),
                 "cols": features(8192), "vectors": rng.randint(1, 96), "master": rng.random() < 0.5}
            if c["weights"] * c["rows"] * c["cols"] + c["vectors"] * c["cols"] <= MOST_VALUES:
                return c
        else:
            c = {"op": op, "M": size(1, 64), "D": features(4096), "F": features(8192), "E": size(2, 128),
                 "act": rng.choice(ACTS[1:]), "gated": rng.random() < 0.6, "bias": rng.random() < 0.4,
                 "residual": rng.random() < 0.5, "normalize": rng.random() < 0.6}
            c["k"] = min(c["E"], size(1, 8))
            if c["E"] * (3 if c["gated"] else 2) * c["D"] * c["F"] <= MOST_EXPERTS_VALUES:
                return c


# -------------------------------------------------------------------- the inputs

def _normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).half()


def _stream(g, m, d):
    """A residual stream: a few columns much larger than the rest, rows away from zero."""
    x = torch.randn((m, d), generator=g, device="cuda", dtype=torch.float32)
    col = torch.rand((d,), generator=g, device="cuda")
    return (x * torch.where(col > 0.99, 6.0, 1.5) + 0.25).half()


def _moments(x, kind):
    x = x.float()
    if kind == 1:
        var, mu = torch.var_mean(x, dim=1, correction=0)
        return mu, torch.rsqrt(var + EPS)
    return torch.zeros(x.shape[0], device="cuda"), torch.rsqrt(x.square().mean(dim=1) + EPS)


def _tensor_sizes(c):
    """How many values each tensor has and where it starts in the program's flat buffers, whole groups apart."""
    sizes = [c["rows"] * c["cols"]] * c["weights"] + [c["cols"]] * c["vectors"]
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // GROUP) * GROUP
    return sizes, starts, total


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]
    s = {"case": case}
    f16 = {"device": "cuda", "dtype": torch.float16}
    f32 = {"device": "cuda", "dtype": torch.float32}
    if op == "residual_norm":
        m, d = c["M"], c["D"]
        s["post"], s["pre"] = NORMS.index(c["post"]), NORMS.index(c["pre"])
        for name, kind in (("post", s["post"]), ("pre", s["pre"])):
            s[name + "_gamma"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")).half() if kind else None
            s[name + "_beta"] = _normal(g, (d,), 0.1) if kind == 1 else None
        s["gate"] = (0.5 + 0.2 * torch.randn((d,), generator=g, device="cuda")).half() if c["gate"] else None
        s["y"] = _normal(g, (m, d), 0.7)
        s["stats"] = torch.zeros((4, m), **f32)
        if c["dir"] == "forward":
            s["x"] = _stream(g, m, d)
            s["z"] = torch.empty((m, d), **f16)
            s["h"] = torch.empty((m, d), **f16) if s["pre"] else None
        else:
            s["z"] = _stream(g, m, d)
            for row, x, kind in ((0, s["y"], s["post"]), (2, s["z"], s["pre"])):
                if kind:
                    mu, rstd = _moments(x, kind)
                    s["stats"][row].copy_(mu)
                    s["stats"][row + 1].copy_(rstd)
            s["dz"] = _normal(g, (m, d), 0.05)
            s["dh"] = _normal(g, (m, d), 0.05) if s["pre"] else None
            s["dx"], s["dy"] = torch.empty((m, d), **f16), torch.empty((m, d), **f16)
            for name, given in (("dgate", s["gate"]), ("dpost_gamma", s["post_gamma"]), ("dpost_beta", s["post_beta"]),
                                ("dpre_gamma", s["pre_gamma"]), ("dpre_beta", s["pre_beta"])):
                s[name] = torch.empty((d,), **f32) if given is not None else None
            # the backward pass's scratch: four rows of partial sums for each of up to 160 groups of rows
            s["work"] = torch.empty((160 * 4 * (d + 32),), **f32)
    elif op == "adamw":
        sizes, starts, total = _tensor_sizes(c)
        inside = torch.zeros(total, device="cuda")
        for n, at in zip(sizes, starts):
            inside[at:at + n] = 1
        # gradients and states of tensors whose groups differ in size, as layers and columns do
        spread = torch.exp(torch.randn((total // GROUP, 1), generator=g, device="cuda"))
        each = torch.exp(0.7 * torch.randn((total // GROUP, GROUP), generator=g, device="cuda")) * spread

        def values(scale):
            x = torch.randn((total // GROUP, GROUP), generator=g, device="cuda")
            return (x * each).reshape(-1) * (inside * scale)

        s["sizes"], s["starts"], s["total"] = sizes, starts, total
        s["decay"] = [DECAY] * c["weights"] + [0.0] * c["vectors"]
        p = values(0.02) / each.reshape(-1)
        s["weight"] = p.half()
        s["master"] = p if c["master"] else None
        s["grad"] = values(0.02).half()
        m, v = values(0.01), values(0.02).square()
        if c["bits"] == 8:
            s["m"], s["m_scales"] = _keep_m(m)
            s["v"], s["v_scales"] = _keep_v(v)
            s["m_out"], s["v_out"] = torch.empty(total, **f32), torch.empty(total, **f32)
        else:
            s["m"], s["v"], s["m_scales"], s["v_scales"] = m, v, None, None
        # each value's decay, by its tensor
        s["keep_rate"] = torch.ones(total, device="cuda")
        for n, at, wd in zip(sizes, starts, s["decay"]):
            s["keep_rate"][at:at + n] = 1 - LR * wd
        s["plan"] = None
    else:
        m, d, f, e = c["M"], c["D"], c["F"], c["E"]
        up = 2 * f if c["gated"] else f
        s["act"] = ACTS.index(c["act"])
        s["x"] = _normal(g, (m, d))
        s["wr"] = _normal(g, (e, d), 2 / math.sqrt(d))
        s["w1"], s["w2"] = _normal(g, (e, up, d), 1 / math.sqrt(d)), _normal(g, (e, d, f), 1 / math.sqrt(f))
        s["b1"], s["b2"] = (_normal(g, (e, up), 0.1), _normal(g, (e, d), 0.1)) if c["bias"] else (None, None)
        s["r"] = _normal(g, (m, d), 2.0) if c["residual"] else None
        s["y"] = torch.empty((m, d), **f16)
        s["chosen"] = torch.empty((m, c["k"]), device="cuda", dtype=torch.int32)
        s["share"] = torch.empty((m, c["k"]), **f32)
        s["work"] = None
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


def _norm(v, kind, gamma, beta):
    """(N(v), μ, ρ) of rows in 32 bits."""
    if kind == 1:
        mu = v.mean(dim=1, keepdim=True)
        c = v - mu
    else:
        mu, c = torch.zeros_like(v[:, :1]), v
    rstd = 1 / torch.sqrt(c.square().mean(dim=1, keepdim=True) + EPS)
    n = c * rstd * gamma.float()
    return (n if beta is None else n + beta.float()), mu[:, 0], rstd[:, 0]


def _norm_back(g, vh, rstd, kind):
    """The gradient of v from that of v̂ = (v − μ)·ρ."""
    along = g - vh * (g * vh).mean(dim=1, keepdim=True)
    return rstd * (along - g.mean(dim=1, keepdim=True) if kind == 1 else along)


def _plain_norm(s):
    c = s["case"]
    y = s["y"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    out = {}
    if c["dir"] == "forward":
        n = y
        if s["post"]:
            n, out["post_mean"], out["post_rstd"] = _norm(y, s["post"], s["post_gamma"], s["post_beta"])
        z = c["alpha"] * s["x"].float() + gate * n
        out["z"] = z.half()
        if s["pre"]:
            h, out["pre_mean"], out["pre_rstd"] = _norm(z, s["pre"], s["pre_gamma"], s["pre_beta"])
            out["h"] = h.half()
        return out
    dz = s["dz"].float()
    if s["pre"]:
        dh, rstd = s["dh"].float(), s["stats"][3][:, None]
        zh = (s["z"].float() - s["stats"][2][:, None]) * rstd
        dz = dz + _norm_back(dh * s["pre_gamma"].float(), zh, rstd, s["pre"])
        out["dpre_gamma"] = (dh * zh).sum(dim=0)
        if s["pre_beta"] is not None:
            out["dpre_beta"] = dh.sum(dim=0)
    out["dx"] = (c["alpha"] * dz).half()
    dn = gate * dz
    n = y
    if s["post"]:
        rstd = s["stats"][1][:, None]
        yh = (y - s["stats"][0][:, None]) * rstd
        n = yh * s["post_gamma"].float()
        out["dpost_gamma"] = (dn * yh).sum(dim=0)
        if s["post_beta"] is not None:
            n = n + s["post_beta"].float()
            out["dpost_beta"] = dn.sum(dim=0)
        out["dy"] = _norm_back(dn * s["post_gamma"].float(), yh, rstd, s["post"]).half()
    else:
        out["dy"] = dn.half()
    if s["gate"] is not None:
        out["dgate"] = (dz * n).sum(dim=0)
    return out


def _keep_m(m):
    """m (32 bits, whole groups) into whole numbers and scales."""
    m = m.view(-1, GROUP)
    top = m.abs().amax(dim=1, keepdim=True)
    zero = top < 2.0 ** -100
    # (tensors on both sides: a number's quotient is computed by its reciprocal)
    most = torch.full_like(top, 127.0)
    q = torch.round(m * torch.where(zero, torch.zeros_like(top), most / top))
    return q.to(torch.int8).view(-1), torch.where(zero, torch.zeros_like(top), top / most).view(-1)


def _keep_v(v):
    """v (32 bits, not negative, whole groups) into 8-bit floats and scales."""
    v = v.view(-1, GROUP)
    top = v.amax(dim=1, keepdim=True)
    zero = top < 2.0 ** -100
    r = v * torch.where(zero, torch.zeros_like(top), torch.ones_like(top) / top)
    code = (255 + ((r.view(torch.int32) - 0x3F800000 + 0x80000) >> 20)).clamp(1, 255)
    code = torch.where(r > 0, code, torch.zeros_like(code))
    return code.to(torch.uint8).view(-1), torch.where(zero, torch.zeros_like(top), top).view(-1)


def _kept_m(codes, scales):
    return (codes.view(-1, GROUP).float() * scales[:, None]).view(-1)


def _kept_v(codes, scales):
    c = codes.view(-1, GROUP).to(torch.int32)
    r = (0x3F800000 + ((c - 255) << 20)).view(torch.float32)
    return (torch.where(c > 0, r, torch.zeros_like(r)) * scales[:, None]).view(-1)


def _plain_adamw(s):
    c = s["case"]
    g = s["grad"].float()
    eight = c["bits"] == 8
    m = (_kept_m(s["m"], s["m_scales"]) if eight else s["m"]) * BETA1 + g * (1 - BETA1)
    v = (_kept_v(s["v"], s["v_scales"]) if eight else s["v"]) * BETA2 + (g * g) * (1 - BETA2)
    p = s["master"] if s["master"] is not None else s["weight"].float()
    step = (m * (LR / (1 - BETA1 ** STEP))) / (torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** STEP)) + ADAM_EPS)
    p = p * s["keep_rate"] - step
    s["weight"].copy_(p)
    out = {"weight": s["weight"]}
    if s["master"] is not None:
        s["master"].copy_(p)
        out["master"] = s["master"]
    if eight:
        for name, keep, kept, x in (("m", _keep_m, _kept_m, m), ("v", _keep_v, _kept_v, v)):
            codes, scales = keep(x)
            s[name].copy_(codes)
            s[name + "_scales"].copy_(scales)
            out[name] = kept(s[name], s[name + "_scales"])
        return out
    s["m"].copy_(m)
    s["v"].copy_(v)
    return {**out, "m": s["m"], "v": s["v"]}


def _choose(logits, k, normalize):
    """The k largest of each row, ties to the lowest index, and their shares."""
    at = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
    share = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    picked = share.gather(1, at)
    return at, picked / (picked if normalize else share).sum(dim=1, keepdim=True)


def _plain_experts(s):
    c = s["case"]
    m, f, e, k = c["M"], c["F"], c["E"], c["k"]
    # next to a border between two experts 32 bits would not do
    at, share = _choose(s["x"].double() @ s["wr"].double().t(), k, c["normalize"])
    share = share.float()
    x = s["x"].float()
    b1, b2 = s["b1"], s["b2"]
    if m * k < e:  # a weight per choice
        pick = at.reshape(-1)
        w1, w2 = s["w1"][pick].float(), s["w2"][pick].float()
        rows = x[:, None, :].expand(m, k, -1).reshape(m * k, 1, -1)
        b1 = None if b1 is None else b1[pick].float()[:, None, :]
        b2 = None if b2 is None else b2[pick].float()[:, None, :]
    else:          # all tokens through every expert
        w1, w2 = s["w1"].float(), s["w2"].float()
        rows = x[None].expand(e, m, -1)
        b1 = None if b1 is None else b1.float()[:, None, :]
        b2 = None if b2 is None else b2.float()[:, None, :]
    u = rows @ w1.transpose(1, 2)
    if b1 is not None:
        u = u + b1
    h = _act(u[..., :f], s["act"]) * u[..., f:] if c["gated"] else _act(u, s["act"])
    o = h @ w2.transpose(1, 2)
    if b2 is not None:
        o = o + b2
    if m * k < e:
        y = (o.view(m, k, -1) * share[:, :, None]).sum(dim=1)
    else:
        full = torch.zeros((m, e), device="cuda").scatter_(1, at, share)
        y = (o * full.t()[:, :, None]).sum(dim=0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.half(), "chosen": at.to(torch.int32), "share": share}


# ------------------------------------------------------------ the library's calls

def _library_norm(s):
    import tensor_core_dense_fp16_gb300 as tc
    c = s["case"]
    m, d = c["M"], c["D"]
    out = {}
    if c["dir"] == "forward":
        tc.hgemm_residual_norm_forward(s["x"], d, c["alpha"], s["y"], d, s["gate"], s["post"], s["post_gamma"],
                                       s["post_beta"], s["pre"], s["pre_gamma"], s["pre_beta"], EPS, s["z"], d, s["h"],
                                       d, s["stats"], m, d)
        out["z"] = s["z"]
        if s["post"]:
            out["post_mean"], out["post_rstd"] = s["stats"][0], s["stats"][1]
        if s["pre"]:
            out["h"], out["pre_mean"], out["pre_rstd"] = s["h"], s["stats"][2], s["stats"][3]
        return out
    tc.hgemm_residual_norm_backward(s["dz"], d, s["dh"], d, s["z"], d, s["y"], d, c["alpha"], s["gate"], s["post"],
                                    s["post_gamma"], s["post_beta"], s["pre"], s["pre_gamma"], s["stats"], s["dx"], d,
                                    s["dy"], d, s["dgate"], s["dpost_gamma"], s["dpost_beta"], s["dpre_gamma"],
                                    s["dpre_beta"], s["work"], m, d)
    return {n: s[n] for n in ("dx", "dy", "dgate", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")
            if s[n] is not None}


def _library_adamw(s):
    import tensor_core_dense_fp16_gb300 as tc
    c = s["case"]
    eight = c["bits"] == 8
    if s["plan"] is None:  # the table that a training program makes once for its tensors
        def part(x, at, n, per=1):
            return None if x is None else x[at // per:at // per + -(-n // per)]
        s["plan"] = tc.hgemm_adamw_tensors([
            dict(weight=part(s["weight"], at, n), master=part(s["master"], at, n), grad=part(s["grad"], at, n),
                 m=part(s["m"], at, n), v=part(s["v"], at, n), m_scales=part(s["m_scales"], at, n, GROUP),
                 v_scales=part(s["v_scales"], at, n, GROUP), weight_decay=wd)
            for n, at, wd in zip(s["sizes"], s["starts"], s["decay"])])
    tc.hgemm_adamw(s["plan"], LR, BETA1, BETA2, ADAM_EPS, STEP)
    out = {"weight": s["weight"]}
    if s["master"] is not None:
        out["master"] = s["master"]
    if eight:
        tc.hgemm_adamw_load(s["m"], s["m_scales"], s["v"], s["v_scales"], s["m_out"], s["v_out"], s["total"])
        return {**out, "m": s["m_out"], "v": s["v_out"]}
    return {**out, "m": s["m"], "v": s["v"]}


def _library_experts(s):
    import tensor_core_dense_fp16_gb300 as tc
    c = s["case"]
    m, d, f, e, k = c["M"], c["D"], c["F"], c["E"], c["k"]
    if s["work"] is None:  # the workspace that a serving program keeps
        s["work"] = torch.empty(tc.hgemm_experts_workspace_size(m, d, f, e, k), device="cuda", dtype=torch.uint8)
    tc.hgemm_experts(s["x"], d, s["wr"], d, s["w1"], d, s["b1"], s["w2"], f, s["b2"], s["act"], c["gated"], k,
                     c["normalize"], s["r"], d, s["y"], d, s["chosen"], s["share"], s["work"], m, d, f, e)
    return {"y": s["y"], "chosen": s["chosen"], "share": s["share"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"residual_norm": _library_norm, "adamw": _library_adamw, "experts": _library_experts}[op](state)
    return {"residual_norm": _plain_norm, "adamw": _plain_adamw, "experts": _plain_experts}[op](state)


# ------------------------------------------------------------- the work of a pass

def work(case):
    c, op = case, case["op"]
    if op == "residual_norm":
        m, d = c["M"], c["D"]
        post, pre = c["post"] != "none", c["pre"] != "none"
        vectors = c["gate"] + post + (c["post"] == "layer") + pre + (c["pre"] == "layer")
        rows = 8 * m * (post + pre)
        if c["dir"] == "forward":
            return {"bytes": (6 + 2 * pre) * m * d + 2 * vectors * d + rows, "flops": m * d * (3 + 6 * post + 6 * pre)}
        # what goes back needs y for its gate's and its norm's gradient, z for the norm's in front
        return {"bytes": (2 + 4 * pre + 2 * (post or c["gate"]) + 4) * m * d + 6 * vectors * d + rows,
                "flops": m * d * (4 + 14 * post + 12 * pre + 2 * c["gate"])}
    if op == "adamw":
        n = c["weights"] * c["rows"] * c["cols"] + c["vectors"] * c["cols"]
        by = 2 + (2 + 8 if c["master"] else 4)
        # 8 bits: codes and scales read and written, then read and written as the values they stand for
        by += 4 + 16 / GROUP + 2 + 8 / GROUP + 8 if c["bits"] == 8 else 16
        return {"bytes": by * n, "flops": 16 * n}
    m, d, f, e, k = c["M"], c["D"], c["F"], c["E"], c["k"]
    # the experts that m tokens are expected to choose, each weight once
    used = min(m * k, e * (1 - (1 - k / e) ** m))
    rows = 3 if c["gated"] else 2
    by = 2 * (used * rows * d * f + e * d + m * d * (3 if c["residual"] else 2)) + 8 * m * k
    if c["bias"]:
        by += 2 * used * ((rows - 1) * f + d)
    return {"bytes": by, "flops": 2 * m * (k * rows * d * f + e * d)}


# ----------------------------------------------------------------- in 64 bits

def _act64(u, name):
    if name == "relu":
        return torch.relu(u)
    if name == "gelu":  # u·σ(2z), z the tanh's argument
        return u * torch.sigmoid(math.sqrt(8 / math.pi) * (u + 0.044715 * u.pow(3)))
    if name == "silu":
        return u * torch.sigmoid(u)
    if name == "gelu_erf":  # u·Φ(u)
        return u * 0.5 * torch.erfc(-u / math.sqrt(2))
    return u * 1


def _double(x):
    return None if x is None else x.double()


def _norm64(v, kind, gamma, beta):
    mu = torch.einsum("md->m", v)[:, None] / v.shape[1] if kind == "layer" else 0.0 * v[:, :1]
    power = torch.einsum("md,md->m", v - mu, v - mu)[:, None] / v.shape[1]
    rstd = (power + EPS).rsqrt()
    n = (v - mu) * rstd * gamma
    return (n if beta is None else n + beta), mu[:, 0], rstd[:, 0]


def _exact_norm(s):
    c = s["case"]
    m, d = c["M"], c["D"]
    y = s["y"].double()
    gate = torch.ones(d, device="cuda", dtype=torch.float64) if s["gate"] is None else s["gate"].double()
    pg, pb, qg, qb = (_double(s[n]) for n in ("post_gamma", "post_beta", "pre_gamma", "pre_beta"))
    out = {}
    if c["dir"] == "forward":
        n = y
        if c["post"] != "none":
            n, out["post_mean"], out["post_rstd"] = _norm64(y, c["post"], pg, pb)
        z = torch.addcmul(c["alpha"] * s["x"].double(), n, gate.expand(m, d))
        out["z"] = z
        if c["pre"] != "none":
            out["h"], out["pre_mean"], out["pre_rstd"] = _norm64(z, c["pre"], qg, qb)
        return out

    def projected(g, vh, kind):
        """g without its parts along v̂ and, of a layer norm, along 1."""
        r = g - vh * (torch.einsum("md,md->m", g, vh) / d)[:, None]
        return r - (torch.einsum("md->m", g) / d)[:, None] if kind == "layer" else r

    dz = s["dz"].double()
    if c["pre"] != "none":
        dh, rho = s["dh"].double(), s["stats"][3].double()[:, None]
        zh = (s["z"].double() - s["stats"][2].double()[:, None]) * rho
        out["dpre_gamma"] = torch.einsum("md,md->d", dh, zh)
        if qb is not None:
            out["dpre_beta"] = torch.einsum("md->d", dh)
        dz = dz + rho * projected(dh * qg, zh, c["pre"])
    out["dx"] = dz * c["alpha"]
    if c["post"] == "none":
        out["dy"] = dz * gate
        if s["gate"] is not None:
            out["dgate"] = torch.einsum("md,md->d", dz, y)
        return out
    rho = s["stats"][1].double()[:, None]
    yh = (y - s["stats"][0].double()[:, None]) * rho
    along, plain = torch.einsum("md,md->d", dz, yh), torch.einsum("md->d", dz)
    out["dpost_gamma"] = gate * along
    if pb is not None:
        out["dpost_beta"] = gate * plain
    if s["gate"] is not None:
        out["dgate"] = pg * along + (0 if pb is None else pb * plain)
    out["dy"] = rho * projected(dz * (gate * pg), yh, c["post"])
    return out


def _exact_adamw(s):
    c = s["case"]
    m, v = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = m * s["m_scales"].double().repeat_interleave(GROUP)
        code = s["v"].double() - 255  # eight to a doubling: 255 − 8j stands for 2^-j
        power = torch.floor(code / 8)
        v = torch.where(s["v"] == 0, 0.0, torch.exp2(power) * (1 + (code / 8 - power)))
        v = v * s["v_scales"].double().repeat_interleave(GROUP)
    g = s["grad"].double()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g.square(), v, BETA2)
    p = (s["master"] if c["master"] else s["weight"]).double()
    rate = torch.zeros_like(p)
    for n, at, wd in zip(s["sizes"], s["starts"], s["decay"]):
        rate[at:at + n] = LR * wd
    p = p - rate * p - LR * (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + ADAM_EPS)
    out = {"weight": p, **({"master": p} if c["master"] else {}), "m": m, "v": v}
    # what 8 bits stand for is a choice of the form's, up to its own steps
    return {**out, "m": None, "v": None} if c["bits"] == 8 else out


def _exact_experts(s):
    c = s["case"]
    m, f, k = c["M"], c["F"], c["k"]
    x = s["x"].double()
    logits = torch.einsum("md,ed->me", x, s["wr"].double())
    order = torch.sort(-logits, dim=1, stable=True)[1][:, :k]
    share = torch.softmax(logits, dim=1).gather(1, order)
    if c["normalize"]:
        share = share / torch.einsum("mk->m", share)[:, None]
    y = s["r"].double() if s["r"] is not None else torch.zeros((m, c["D"]), device="cuda", dtype=torch.float64)
    for e in range(c["E"]):
        token, slot = (order == e).nonzero(as_tuple=True)
        if not len(token):
            continue
        u = torch.einsum("td,fd->tf", x[token], s["w1"][e].double())
        if s["b1"] is not None:
            u += s["b1"][e].double()
        h = _act64(u[:, :f], c["act"])
        if c["gated"]:
            h = h * u[:, f:]
        o = torch.einsum("tf,df->td", h, s["w2"][e].double())
        if s["b2"] is not None:
            o += s["b2"][e].double()
        y = y.index_add(0, token, o * share[token, slot][:, None])
    return {"y": y, "chosen": None, "share": share}


def exact(case, seed):
    """Each output before its rounding to 16 bits."""
    s = prepare(case, seed)
    return {"residual_norm": _exact_norm, "adamw": _exact_adamw, "experts": _exact_experts}[case["op"]](s)
