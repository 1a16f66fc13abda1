"""The experts' layer against the 64-bit reference, within the bounds
around_reference derives (GPU only)."""

import numpy as np
import pytest

import around_reference as ref
import block_reference
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import Matrix, check, done, rng_half

pytestmark = pytest.mark.gpu


def make(m, d, f, e, gated, bias, res, seed=0):
    rng = np.random.default_rng(seed + 7 * m + d + f + e)
    up = 2 * f if gated else f
    return {"x": rng_half(rng, (m, d)), "wr": rng_half(rng, (e, d), 2 / max(1, d) ** 0.5),
            "w1": rng_half(rng, (e, up, d), 1 / max(1, d) ** 0.5), "w2": rng_half(rng, (e, d, f), 1 / max(1, f) ** 0.5),
            "b1": rng_half(rng, (e, up), 0.3) if bias else None, "b2": rng_half(rng, (e, d), 0.3) if bias else None,
            "r": rng_half(rng, (m, d), 2) if res else None}


def call(v, act, gated, k, normalize, pad=0, offset=0, in_place=False, wanted=True, stream=None):
    """(y, chosen, share) as the kernels leave them."""
    torch = torch_cuda()
    m, d = v["x"].shape
    e, _, f = v["w2"].shape
    up = v["w1"].shape[1]

    def matrix(a, rows, cols, p=pad):
        return None if a is None else Matrix(rows, cols, cols + p, offset, value=a.reshape(rows, cols))

    X, WR, W1 = matrix(v["x"], m, d), matrix(v["wr"], e, d), matrix(v["w1"], e * up, d)
    W2, R = matrix(v["w2"], e * d, f), matrix(v["r"], m, d)
    B1, B2 = matrix(v["b1"], 1, e * up, 0), matrix(v["b2"], 1, e * d, 0)
    Y = R if in_place else Matrix(m, d, d + pad, offset)
    C = Matrix(m, k, dtype=np.int32) if wanted else None
    S = Matrix(m, k, dtype=np.float32) if wanted else None
    size = tc.hgemm_experts_workspace_size(m, d, f, e, k)
    work = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    p = lambda t: None if t is None else t.ptr  # noqa: E731
    tc.hgemm_experts(X.ptr, X.ld, WR.ptr, WR.ld, W1.ptr, W1.ld, p(B1), W2.ptr, W2.ld, p(B2),
                     block_reference.ACTS.index(act), gated, k, normalize, p(R), R.ld if R else 0, Y.ptr, Y.ld, p(C),
                     p(S), work, m, d, f, e, workspace_bytes=size, stream=stream)
    done()
    assert (work[size:] == 255).all(), "written behind the workspace"
    return Y.get(), C.get() if C else None, S.get() if S else None


def run(m, d, f, e, k, act="silu", gated=True, bias=False, res=True, normalize=True, seed=0, **how):
    v = make(m, d, f, e, gated, bias, res, seed)
    y, chosen, share = call(v, act, gated, k, normalize, **how)
    if chosen is None:
        _, chosen, share = call(v, act, gated, k, normalize)
    what = f"{m} tokens {d}->{f}, {k} of {e}, {act} "
    assert ((chosen >= 0) & (chosen < e)).all()
    logits, el, s, es, want, bound = ref.experts(v["x"], v["wr"], v["w1"], v["b1"], v["w2"], v["b2"], act, gated,
                                                 normalize, v["r"], chosen)
    # the choice: different experts, from the largest logit down, none larger left out, up to the logits' errors
    for i in range(m):
        assert len(set(chosen[i])) == k, what
        l, err = logits[i], el[i]
        mine = l[chosen[i]]
        assert (mine[:-1] >= mine[1:] - 2 * err.max()).all(), what + "order"
        left = np.delete(l, chosen[i])
        assert left.size == 0 or left.max() <= mine.min() + 2 * err.max(), what + "largest"
    check(share, s, es, what + "share")
    check(y, want, bound, what + "y")


SHAPES = [(1, 64, 64, 2, 1), (1, 2048, 512, 8, 2), (1, 72, 4104, 4, 4), (2, 65, 7, 3, 2), (7, 264, 200, 10, 3),
          (8, 512, 256, 16, 8), (9, 128, 1024, 5, 5), (16, 1000, 72, 64, 4), (17, 136, 136, 33, 6), (24, 256, 512, 64, 8),
          (33, 77, 131, 12, 2), (64, 256, 264, 8, 2), (64, 64, 64, 1, 1), (64, 40, 24, 512, 16), (3, 1, 1, 2, 2),
          (5, 8200, 8, 4, 2), (40, 1024, 2056, 3, 2)]


@pytest.mark.parametrize("m,d,f,e,k", SHAPES)
@pytest.mark.parametrize("gated", [True, False])
def test_shapes(m, d, f, e, k, gated):
    run(m, d, f, e, k, gated=gated, bias=not gated)


@pytest.mark.parametrize("act", block_reference.ACTS)
@pytest.mark.parametrize("gated,bias,res,normalize", [(True, True, False, False), (False, False, True, True),
                                                      (True, False, True, False)])
@pytest.mark.parametrize("m", [1, 20])
def test_epilogues(act, gated, bias, res, normalize, m):
    run(m, 136, 200, 9, 3, act, gated, bias, res, normalize)


@pytest.mark.parametrize("m", [1, 12])
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4)])
def test_pitches_and_alignment(m, pad, offset):
    run(m, 136, 72, 6, 2, bias=True, pad=pad, offset=offset)


def test_in_place_and_without_the_choice():
    run(10, 264, 136, 6, 2, in_place=True)
    run(10, 264, 136, 6, 2, wanted=False)
    run(10, 264, 136, 6, 2, stream=torch_cuda().cuda.Stream())


def test_no_tokens_and_empty_sizes():
    run(3, 64, 0, 4, 2, bias=True)
    v = make(1, 64, 8, 4, True, False, False)
    v["x"] = v["x"][:0]
    y, chosen, share = call(v, "silu", True, 2, True)
    assert y.shape == (0, 64) and chosen.shape == (0, 2)


def test_ties_go_to_the_lowest_index():
    """Logits that are small whole numbers, exact in FP32."""
    torch = torch_cuda()
    d, e, k = 64, 40, 5
    rng = np.random.default_rng(2)
    v = make(30, d, 16, e, True, False, False)
    v["x"] = np.zeros((30, d), np.float16)
    v["x"][:, :8] = rng.integers(-2, 3, (30, 8))
    v["wr"] = np.zeros((e, d), np.float16)
    v["wr"][:, :8] = rng.integers(-1, 2, (e, 8))
    v["x"][0] = 0  # all logits 0: the first k
    _, chosen, _ = call(v, "silu", True, k, True)
    logits = v["x"].astype(np.float64) @ v["wr"].astype(np.float64).T
    want = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    assert (chosen == want).all()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("normalize", [True, False])
def test_nan_and_infinities_stay_in_their_tokens(normalize):
    v = make(12, 136, 72, 6, True, True, True)
    clean = call(v, "silu", True, 2, normalize)
    x = v["x"].copy()
    x[3, 5], x[7, 0], x[9, 100] = np.nan, np.inf, -np.inf
    y, chosen, share = call({**v, "x": x}, "silu", True, 2, normalize)
    rows = [i for i in range(12) if i not in (3, 7, 9)]
    assert (chosen[rows] == clean[1][rows]).all() and (share[rows] == clean[2][rows]).all()
    assert (y[rows] == clean[0][rows]).all()
    assert ((chosen >= 0) & (chosen < 6)).all()
    assert (chosen[3] == [0, 1]).all(), "all logits NaN: the lowest"
    assert np.isnan(y[3]).all()
    # an expert whose weights hold a NaN spoils those who chose it alone
    w1 = v["w1"].copy()
    bad = int(clean[1][0, 0])
    w1[bad, 3, 7] = np.nan
    y, _, _ = call({**v, "w1": w1}, "silu", True, 2, normalize)
    hit = (clean[1] == bad).any(axis=1)
    assert np.isnan(y[hit]).all() and (y[~hit] == clean[0][~hit]).all()


def test_a_nan_logit_is_below_every_number():
    v = make(4, 64, 16, 5, True, False, False)
    wr = v["wr"].copy()
    wr[2, 3] = np.nan
    _, chosen, share = call({**v, "wr": wr}, "silu", True, 4, True)
    assert (chosen != 2).all() and np.isfinite(share).all()
    wr[4] = 0
    wr[4, 0] = -np.inf
    v["x"][:, 0] = 1
    _, chosen, _ = call({**v, "wr": wr}, "silu", True, 5, True)
    assert (chosen[:, 3] == 4).all() and (chosen[:, 4] == 2).all()


def test_all_tokens_on_one_expert_and_on_all():
    for wr in (1, 0):
        v = make(64, 128, 256, 4, True, False, True)
        if wr:
            v["x"][:, 0] = 1
            v["wr"][:] = 0
            v["wr"][2, 0] = 5
        y, chosen, share = call(v, "silu", True, 1 if wr else 4, True)
        assert (chosen[:, 0] == 2).all() or not wr
        want = ref.experts(v["x"], v["wr"], v["w1"], None, v["w2"], None, "silu", True, True, v["r"], chosen)
        check(y, want[4], want[5], "y")


def test_equal_calls_give_equal_bits_and_replay():
    torch = torch_cuda()
    m, d, f, e, k = 24, 512, 264, 16, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).half()  # noqa: E731
    x, wr, w1, w2 = n(m, d), n(e, d) * 4, n(e, 2 * f, d), n(e, d, f)
    y, c, s = torch.empty_like(x), torch.empty(m, k, dtype=torch.int32, device="cuda"), torch.empty(m, k, device="cuda")
    work = torch.empty(tc.hgemm_experts_workspace_size(m, d, f, e, k), dtype=torch.uint8, device="cuda")

    def layer():
        tc.hgemm_experts(x, d, wr, d, w1, d, None, w2, f, None, 3, True, k, True, x, d, y, d, c, s, work, m, d, f, e)

    layer()
    torch.cuda.synchronize()
    want = y.clone(), c.clone(), s.clone()
    for _ in range(3):
        work.fill_(255)
        layer()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(c, want[1]) and torch.equal(s, want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer()
            layer()
    # other tokens in the same buffers
    old = x.clone()
    x.copy_(n(m, d))
    graph.replay()
    torch.cuda.synchronize()
    other = y.clone()
    layer()
    torch.cuda.synchronize()
    assert torch.equal(y, other) and not torch.equal(y, want[0])
    x.copy_(old)
    work.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])
    done()


def test_calls_one_after_another_on_one_workspace():
    """Different layers in a row on one stream and one workspace, as a model calls them."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).half()  # noqa: E731
    layers, size = [], 0
    for m, d, f, e, k in ((5, 256, 512, 8, 2), (64, 256, 72, 32, 8), (1, 256, 1024, 4, 1), (20, 256, 77, 6, 3)):
        layers.append((m, d, f, e, k, n(m, d) * 16, n(e, d) * 4, n(e, 2 * f, d), n(e, d, f)))
        size = max(size, tc.hgemm_experts_workspace_size(m, d, f, e, k))
    work = torch.empty(size, dtype=torch.uint8, device="cuda")

    def call_all(each):
        out = []
        for m, d, f, e, k, x, wr, w1, w2 in layers:
            y = torch.empty_like(x)
            w = torch.empty(size, dtype=torch.uint8, device="cuda") if each else work
            tc.hgemm_experts(x, d, wr, d, w1, d, None, w2, f, None, 3, True, k, True, x, d, y, d, None, None, w, m, d, f,
                             e)
            if each:
                torch.cuda.synchronize()
            out.append(y)
        done()
        return out

    want = call_all(True)
    for _ in range(5):
        for a, b in zip(call_all(False), want):
            assert torch.equal(a, b)
