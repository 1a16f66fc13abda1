"""The norms around a block against the 64-bit reference, within the bounds
around_reference derives (GPU only)."""

import numpy as np
import pytest

import around_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import Matrix, check, done, rng_half

pytestmark = pytest.mark.gpu

EPS = 1e-5


def vectors(rng, d, offset, post, pre, gate, beta):
    """(host, device) vectors; absent ones None."""
    def one(there, value):
        if not there:
            return None, None
        v = value.astype(np.float16)
        return v, Matrix(1, d, offset=offset, value=v[None, :])
    std = rng.standard_normal
    return {"gate": one(gate, 0.5 + 0.3 * std(d)),
            "post_gamma": one(post != "none", 1 + 0.2 * std(d)), "post_beta": one(post != "none" and beta, 0.2 * std(d)),
            "pre_gamma": one(pre != "none", 1 + 0.2 * std(d)), "pre_beta": one(pre != "none" and beta, 0.2 * std(d))}


def ptr(m):
    return None if m is None else m.ptr


def values(rng, m, d):
    """Rows off zero, some columns large, one row constant and one of zeros."""
    x = rng.standard_normal((m, d)) * np.where(rng.random(d) > 0.98, 6, 1) + rng.standard_normal((m, 1))
    if m > 3:
        x[1] = 0.5
        x[2] = 0
    return x.astype(np.float16)


def check16(got, want, bound, what):
    """check, for FP16: from 65520 on, halfway between the largest FP16 value
    and the next step, a value rounds to infinity, and only from there on."""
    got = got.astype(np.float64)
    over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= 65520)
    check(np.where(over, want, got), want, bound, what)


def run_forward(m, d, post="rms", pre="rms", gate=True, beta=True, alpha=1.0, pad=0, offset=0, in_place=False,
                stats=True, seed=0, stream=None):
    rng = np.random.default_rng(seed + 13 * m + d)
    x, y = values(rng, m, d), values(rng, m, d)
    v = vectors(rng, d, offset, post, pre, gate, beta)
    X, Y = Matrix(m, d, d + pad, offset, value=x), Matrix(m, d, d + pad, offset, value=y)
    Z = X if in_place else Matrix(m, d, d + pad, offset)
    H = None if pre == "none" else Y if in_place else Matrix(m, d, d + pad, offset)
    S = Matrix(4, m, dtype=np.float32) if stats else None
    kinds = [ref.NORMS.index(post), ref.NORMS.index(pre)]
    tc.hgemm_residual_norm_forward(X.ptr, X.ld, alpha, Y.ptr, Y.ld, ptr(v["gate"][1]), kinds[0],
                                   ptr(v["post_gamma"][1]), ptr(v["post_beta"][1]), kinds[1], ptr(v["pre_gamma"][1]),
                                   ptr(v["pre_beta"][1]), EPS, Z.ptr, Z.ld, ptr(H), H.ld if H else 0, ptr(S), m, d,
                                   stream)
    done()
    want = ref.residual_norm(x, alpha, y, v["gate"][0], post, v["post_gamma"][0], v["post_beta"][0], pre,
                             v["pre_gamma"][0], v["pre_beta"][0], EPS)
    what = f"{m}x{d} {post} {pre} pad {pad} offset {offset} "
    check16(Z.get(), *want["z"], what + "z")
    if H:
        check16(H.get(), *want["h"], what + "h")
    if S:
        s = S.get()
        for row, name in enumerate(("post_mean", "post_rstd", "pre_mean", "pre_rstd")):
            if name in want:
                check(s[row], *want[name], what + name)
            else:
                assert (s[row] == 77).all(), what + name + " was written"


def run_backward(m, d, post="rms", pre="rms", gate=True, beta=True, alpha=1.0, residual=True, pad=0, offset=0,
                 in_place=False, wanted=True, seed=1, stream=None):
    rng = np.random.default_rng(seed + 13 * m + d)
    z, y = values(rng, m, d), values(rng, m, d)
    dz, dh = rng_half(rng, (m, d), 0.1), rng_half(rng, (m, d), 0.1)
    v = vectors(rng, d, offset, post, pre, gate, beta)
    stats = np.zeros((4, m), np.float32)
    for row, t, kind in ((0, y, post), (2, z, pre)):
        if kind != "none":
            t = t.astype(np.float64)
            mu = t.mean(axis=1) if kind == "layer" else np.zeros(m)
            stats[row], stats[row + 1] = mu, 1 / np.sqrt(((t - mu[:, None]) ** 2).mean(axis=1) + EPS)
    Z, Y = Matrix(m, d, d + pad, offset, value=z), Matrix(m, d, d + pad, offset, value=y)
    DZ = Matrix(m, d, d + pad, offset, value=dz) if residual else None
    DH = Matrix(m, d, d + pad, offset, value=dh) if pre != "none" else None
    DX = DZ if in_place and DZ else Matrix(m, d, d + pad, offset)
    DY = DH if in_place and DH else Matrix(m, d, d + pad, offset)
    S = Matrix(4, m, dtype=np.float32, value=stats)
    there = {"dgate": gate, "dpost_gamma": post != "none", "dpost_beta": post != "none", "dpre_gamma": pre != "none",
             "dpre_beta": pre != "none"}
    G = {n: Matrix(1, d, dtype=np.float32) if t and wanted else None for n, t in there.items()}
    size = tc.hgemm_residual_norm_backward_workspace_size(m, d)
    work = torch_cuda().empty(size, dtype=torch_cuda().uint8, device="cuda")
    tc.hgemm_residual_norm_backward(
        ptr(DZ), DZ.ld if DZ else 0, ptr(DH), DH.ld if DH else 0, Z.ptr, Z.ld, Y.ptr, Y.ld, alpha, ptr(v["gate"][1]),
        ref.NORMS.index(post), ptr(v["post_gamma"][1]), ptr(v["post_beta"][1]), ref.NORMS.index(pre),
        ptr(v["pre_gamma"][1]), S.ptr, DX.ptr, DX.ld, DY.ptr, DY.ld, *(ptr(G[n]) for n in there), work, m, d,
        stream=stream)
    done()
    want = ref.residual_norm_backward(dz if residual else None, dh, z, y, alpha, v["gate"][0], post,
                                      v["post_gamma"][0], v["post_beta"][0], pre, v["pre_gamma"][0], stats)
    what = f"{m}x{d} {post} {pre} pad {pad} offset {offset} "
    check16(DX.get(), *want["dx"], what + "dx")
    check16(DY.get(), *want["dy"], what + "dy")
    for n, t in G.items():
        if t:
            check(t.get()[0], *want[n], what + n)
    S.get(), Z.get(), Y.get()
    return [DX.buf, DY.buf] + [t.buf for t in G.values() if t]


# one value to rows longer than a block holds, on both sides of every change of kernel
SHAPES = [(1, 1), (1, 64), (1, 4096), (2, 7), (3, 8), (5, 513), (70, 264), (33, 1000), (9, 2048), (4, 4104), (3, 8192),
          (2, 8200), (3, 16384), (2, 20001), (700, 128), (1300, 72), (1500, 65), (400, 1024)]
KINDS = [(p, q) for p in ref.NORMS for q in ref.NORMS]


@pytest.mark.parametrize("m,d", SHAPES)
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer")])
def test_shapes(m, d, post, pre):
    run_forward(m, d, post, pre)
    run_backward(m, d, post, pre)


@pytest.mark.parametrize("m,d", [(1, 200), (40, 264), (31, 77)])
@pytest.mark.parametrize("post,pre", KINDS)
@pytest.mark.parametrize("gate,beta,alpha", [(False, False, 1.0), (True, True, 0.75), (False, True, -2.0)])
def test_kinds(m, d, post, pre, gate, beta, alpha):
    run_forward(m, d, post, pre, gate, beta, alpha)
    run_backward(m, d, post, pre, gate, beta, alpha, residual=beta)


@pytest.mark.parametrize("m,d", [(1, 264), (40, 264), (700, 136), (300, 77)])
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4)])
def test_pitches_and_alignment(m, d, pad, offset):
    run_forward(m, d, "layer", "rms", pad=pad, offset=offset)
    run_backward(m, d, "rms", "layer", pad=pad, offset=offset)


@pytest.mark.parametrize("m,d", [(1, 264), (40, 4096), (300, 77), (700, 128), (2, 20001)])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("layer", "none")])
def test_in_place(m, d, post, pre):
    run_forward(m, d, post, pre, in_place=True)
    run_backward(m, d, post, pre, in_place=True)


@pytest.mark.parametrize("d", [264, 77, 8192])
def test_nothing_but_the_rows_is_wanted(d):
    run_forward(40, d, stats=False)
    run_backward(40, d, wanted=False)


def test_more_rows_than_a_pass_of_any_grid():
    run_forward(70000, 8, "layer", "rms")
    run_backward(70000, 8, "layer", "rms")
    run_backward(70000, 9, "layer", "rms")


@pytest.mark.parametrize("m,d", [(3800, 1000), (1900, 1800), (1000, 4096), (1400, 2200), (520, 8192), (200, 16384)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_several_waves_of_rows(m, d, kind):
    """More rows than the GPU holds at once, in rows of every number of threads."""
    run_forward(m, d, kind, kind, pad=8)
    if d <= 8192:
        run_backward(m, d, kind, kind, pad=8)


def test_no_rows():
    torch = torch_cuda()
    h = torch.zeros(64, dtype=torch.float16, device="cuda")
    f = torch.full((3, 64), 5.0, device="cuda")
    work = torch.empty(tc.hgemm_residual_norm_backward_workspace_size(0, 64), dtype=torch.uint8, device="cuda")
    tc.hgemm_residual_norm_backward(None, 0, None, 64, None, 64, None, 64, 1.0, h, 2, h, None, 2, h, None, None, 64,
                                    None, 64, f[0], f[1], None, f[2], None, work, 0, 64)
    done()
    assert (f == 0).all()


@pytest.mark.parametrize("d", [264, 77])
def test_infinities_and_nan_stay_in_their_rows(d):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    x, y = (torch.randn(6, d, generator=g, device="cuda").half() for _ in range(2))
    gamma = torch.ones(d, dtype=torch.float16, device="cuda")
    outs = []
    for spoil in (False, True):
        xs, ys = x.clone(), y.clone()
        if spoil:
            xs[1, 5], ys[2, 7], ys[4, 0] = float("nan"), float("inf"), float("nan")
        z, h = torch.empty_like(x), torch.empty_like(x)
        stats = torch.empty(4, 6, device="cuda")
        tc.hgemm_residual_norm_forward(xs, d, 1.0, ys, d, None, 2, gamma, None, 1, gamma, None, EPS, z, d, h, d, stats,
                                       6, d)
        done()
        outs.append((z, h, stats))
    for a, b in zip(*outs):
        rows = (0, 3, 5)
        if a.shape[0] == 4:
            a, b = a.t(), b.t()
        assert torch.equal(a[rows, :], b[rows, :])
    z, h, _ = outs[1]
    assert h[1].isnan().all() and h[2].isnan().any() and h[4].isnan().all()
    assert not z[1, :5].isnan().any() and z[1, 5].isnan()


@pytest.mark.parametrize("d", [256, 2048, 77, 8192])
def test_equal_calls_give_equal_bits(d):
    torch = torch_cuda()
    a, b = run_backward(900, d, "layer", "layer"), run_backward(900, d, "layer", "layer")
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "layer"), ("rms", "none")])
def test_gradients_against_differences(post, pre):
    """Σ z·dZ + Σ h·dH, evaluated in 64 bits, changes along a direction as the
    gradients say; central differences of step 1e-5 are off by its square times
    the third derivative and by 2^-52/1e-5: 1e-6 of the terms' size, beside the
    FP16 gradients' 2^-11."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(5)
    m, d, alpha = 12, 96, 0.75

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda").half()

    x, y, dz, dh = (normal(m, d) for _ in range(4))
    gate, pg, pb, qg, qb = (normal(d) for _ in range(5))
    if post != "layer":
        pb = None
    if post == "none":
        pg = None
    if pre == "none":
        qg = qb = dh = None
    p, q = ref.NORMS.index(post), ref.NORMS.index(pre)
    z, h = torch.empty_like(x), torch.empty_like(x) if q else None
    stats = torch.zeros(4, m, device="cuda")
    tc.hgemm_residual_norm_forward(x, d, alpha, y, d, gate, p, pg, pb, q, qg, qb, EPS, z, d, h, d, stats, m, d)

    def loss(v):
        def n(t, kind, gamma, beta):
            c = t - t.mean(axis=1, keepdims=True) if kind == "layer" else t
            r = c / np.sqrt((c * c).mean(axis=1, keepdims=True) + EPS)
            return r * gamma + (0 if beta is None else beta)
        zz = alpha * v["x"] + v["gate"] * (v["y"] if post == "none" else n(v["y"], post, v["pg"], v["pb"]))
        total = (zz * num(dz)).sum()
        return total if pre == "none" else total + (n(zz, pre, v["qg"], v["qb"]) * num(dh)).sum()

    def num(t):
        return None if t is None else t.double().cpu().numpy()

    at = {"x": num(x), "y": num(y), "gate": num(gate), "pg": num(pg), "pb": num(pb), "qg": num(qg), "qb": num(qb)}
    f = lambda t: torch.empty(d, device="cuda") if t is not None else None  # noqa: E731
    dx, dy, sums = torch.empty_like(x), torch.empty_like(x), [f(gate), f(pg), f(pb), f(qg), f(qb)]
    work = torch.empty(tc.hgemm_residual_norm_backward_workspace_size(m, d), dtype=torch.uint8, device="cuda")
    tc.hgemm_residual_norm_backward(dz, d, dh, d, z, d, y, d, alpha, gate, p, pg, pb, q, qg, stats, dx, d, dy, d, *sums,
                                    work, m, d)
    done()
    grads = dict(zip(("x", "y", "gate", "pg", "pb", "qg", "qb"), map(num, (dx, dy, *sums))))
    rng = np.random.default_rng(6)
    for name, grad in grads.items():
        if grad is None:
            continue
        for _ in range(3):
            way = rng.standard_normal(grad.shape)
            up, down = ({**at, name: at[name] + s * 1e-5 * way} for s in (1, -1))
            want = (loss(up) - loss(down)) / 2e-5
            # the gradients' and the stored z's roundings are independent of one another: 2^-11 of each
            # term at most, a few terms to a gradient; twelve times that in the 2-norm
            off = abs((grad * way).sum() - want)
            assert off <= 12 * 2.0 ** -11 * np.linalg.norm(grad * way) + 1e-5 * np.abs(grad * way).sum(), name


@pytest.mark.parametrize("d", [264, 77, 8192])
def test_on_another_stream_and_replayed(d):
    torch = torch_cuda()
    side = torch.cuda.Stream()
    run_forward(40, d, "layer", "layer", stream=side)
    run_backward(40, d, "layer", "layer", stream=side)
    g = torch.Generator(device="cuda").manual_seed(5)
    m = 300
    z, y, dz, dh = (torch.randn(m, d, generator=g, device="cuda").half() for _ in range(4))
    gamma = torch.ones(d, dtype=torch.float16, device="cuda")
    stats = torch.rand(4, m, generator=g, device="cuda") + 0.5
    dx, dy, dg = torch.empty_like(z), torch.empty_like(z), torch.empty(2, d, device="cuda")
    work = torch.empty(tc.hgemm_residual_norm_backward_workspace_size(m, d), dtype=torch.uint8, device="cuda")

    def call():
        tc.hgemm_residual_norm_backward(dz, d, dh, d, z, d, y, d, 1.0, None, 1, gamma, None, 2, gamma, stats, dx, d,
                                        dy, d, None, dg[0], None, dg[1], None, work, m, d)

    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dx, dy, dg)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for t in (dx, dy, dg):
        t.zero_()
    work.fill_(255)
    graph.replay()
    done()
    torch.cuda.synchronize()
    for t, w in zip((dx, dy, dg), want):
        assert torch.equal(t, w)
