"""The feed-forward block's operators against the 64-bit reference, within
the bounds block_reference derives (GPU only)."""

import numpy as np
import pytest

import block_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu

GUARD = 77.0  # what lies around an output and must stay


def rng_half(rng, shape, scale=1.0):
    return (rng.standard_normal(shape) * scale).astype(np.float16)


class Matrix:
    """A device matrix with a pitch and an offset inside a larger buffer, guarded all around."""

    def __init__(self, rows, cols, ld=None, offset=0, dtype=np.float16, value=None):
        torch = torch_cuda()
        self.rows, self.cols, self.ld, self.offset = rows, cols, cols if ld is None else ld, offset
        self.n = offset + max(rows, 1) * max(self.ld, 1) + 16
        host = np.full(self.n, GUARD).astype(dtype)
        if value is not None:
            self._view(host)[:] = value
        self.buf = torch.from_numpy(host).to("cuda")

    def _view(self, flat):
        return np.lib.stride_tricks.as_strided(flat[self.offset:], (self.rows, self.cols),
                                               (self.ld * flat.itemsize, flat.itemsize))

    @property
    def ptr(self):
        return self.buf[self.offset:].data_ptr()

    def get(self):
        flat = self.buf.cpu().numpy()
        out = self._view(flat).copy()
        self._view(flat)[:] = np.array(GUARD).astype(flat.dtype)
        assert (flat == np.array(GUARD).astype(flat.dtype)).all(), "written outside the matrix"
        return out


def done():
    assert tc.hgemm_device_status() == tc.HGEMM_OK


def check(got, want, bound, what):
    got = got.astype(np.float64)
    bad = ~(np.abs(got - want) <= bound)
    bad &= ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]}, bound "
                           f"{np.broadcast_to(bound, bad.shape)[bad][0]}")


# pad: extra pitch of every matrix; offset: elements its base is moved by
def run_linear(M, N, K, name, bias=True, res=True, keep=False, pad=0, offset=0, in_place=False, seed=0, stream=None):
    rng = np.random.default_rng(seed + 31 * M + 7 * N + K)
    x, w = rng_half(rng, (M, K)), rng_half(rng, (N, K), 1 / max(1, K) ** 0.5)
    b = rng_half(rng, (1, N)) if bias else None
    r = rng_half(rng, (M, N), 2) if res else None
    X, W = Matrix(M, K, K + pad, offset, value=x), Matrix(N, K, K + pad, offset, value=w)
    B = Matrix(1, N, offset=offset, value=b) if bias else None
    Y = Matrix(M, N, N + pad, offset, value=r if in_place else None)
    R = Y if in_place else (Matrix(M, N, N + pad, offset, value=r) if res else None)
    groups = -(-N // 64)
    Q = Matrix(M, N, N + pad, offset, np.int8) if keep else None
    S = Matrix(groups, M, M + pad, offset, np.float32) if keep else None
    tc.hgemm_linear(X.ptr, X.ld, W.ptr, W.ld, B.ptr if B else None, ref.ACTS.index(name), R.ptr if R else None,
                    R.ld if R else 0, Y.ptr, Y.ld, M, N, K, Q.ptr if Q else None, Q.ld if Q else 0,
                    S.ptr if S else None, S.ld if S else 0, stream)
    done()
    y, ey, u, eu = ref.linear(x, w, b[0] if bias else None, name, r)
    what = f"linear {M}x{N}x{K} {name} pad {pad} offset {offset}"
    check(Y.get(), y, ey, what)
    if keep:
        codes, scales = Q.get(), S.get()
        pu = np.zeros((M, groups * 64))
        pu[:, :N] = np.abs(u)
        pe = np.zeros((M, groups * 64))
        pe[:, :N] = eu
        top, et = pu.reshape(M, groups, 64).max(axis=2).T, pe.reshape(M, groups, 64).max(axis=2).T
        check(scales, top / 127, et / 127 + 2.0 ** -22 * top, what + " scales")
        half = np.repeat(scales.astype(np.float64).T, 64, axis=1)[:, :N] / 2
        check(ref.kept(codes, scales), u, half * (1 + 2.0 ** -14) + eu, what + " codes")


SHAPES = [(1, 64, 64), (1, 1, 1), (2, 7, 65), (1, 2048, 512), (8, 520, 1000), (17, 1000, 264), (33, 4096, 3200),
          (129, 65, 200), (300, 136, 72), (128, 10240, 64), (1000, 1000, 1000), (513, 1032, 200), (64, 512, 8000),
          (2048, 2048, 128), (2500, 2304, 72), (300, 129, 136), (77, 40, 33)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("name", ["gelu", "none"])
def test_linear_shapes(M, N, K, name):
    run_linear(M, N, K, name, keep=name == "gelu")


@pytest.mark.parametrize("M,N,K", [(1, 200, 136), (5, 72, 520), (40, 200, 264), (300, 200, 136)])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True)])
def test_linear_epilogues(M, N, K, name, bias, res):
    run_linear(M, N, K, name, bias=bias, res=res, keep=not res)


@pytest.mark.parametrize("M,N,K", [(1, 200, 136), (20, 136, 520), (300, 200, 264)])
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4)])
def test_linear_pitches_and_alignment(M, N, K, pad, offset):
    run_linear(M, N, K, "silu", keep=True, pad=pad, offset=offset)


@pytest.mark.parametrize("M,N,K", [(1, 264, 72), (30, 264, 72), (300, 264, 72), (300, 131, 71)])
def test_linear_residual_in_place(M, N, K):
    run_linear(M, N, K, "gelu", in_place=True, keep=True)


@pytest.mark.parametrize("M,N", [(1, 65), (130, 200)])
def test_linear_empty_sum(M, N):
    run_linear(M, N, 0, "gelu", keep=True)
    run_linear(M, N, 0, "none", bias=False, res=False)


def run_dgrad(M, N, K, name, hidden=True, pad=0, offset=0, seed=1):
    rng = np.random.default_rng(seed + 31 * M + 7 * N + K)
    dy, w = rng_half(rng, (M, N)), rng_half(rng, (N, K), 1 / max(1, N) ** 0.5)
    codes, scales = ref.keep32((rng.standard_normal((M, K)) * 2).astype(np.float32))
    with_act = name is not None
    DY, W = Matrix(M, N, N + pad, offset, value=dy), Matrix(N, K, K + pad, offset, value=w)
    Q = Matrix(M, K, K + pad, offset, np.int8, codes) if with_act else None
    S = Matrix(scales.shape[0], M, M + pad, offset, np.float32, scales) if with_act else None
    DU = Matrix(M, K, K + pad, offset)
    H = Matrix(M, K, K + pad, offset) if hidden and with_act else None
    tc.hgemm_linear_dgrad(DY.ptr, DY.ld, W.ptr, W.ld, Q.ptr if Q else None, Q.ld if Q else 0,
                          S.ptr if S else None, S.ld if S else 0, ref.ACTS.index(name) if with_act else 0,
                          DU.ptr, DU.ld, H.ptr if H else None, H.ld if H else 0, M, N, K)
    done()
    du, edu, h, eh = ref.dgrad(dy, w, codes if with_act else None, scales, name)
    what = f"dgrad {M}x{N}x{K} {name} pad {pad} offset {offset}"
    check(DU.get(), du, edu, what)
    if H:
        check(H.get(), h, eh, what + " H")


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dgrad_shapes(M, N, K):
    run_dgrad(M, N, K, "gelu")
    run_dgrad(M, N, K, None)


@pytest.mark.parametrize("M,N,K", [(40, 200, 264), (300, 200, 136)])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("hidden", [False, True])
def test_dgrad_activations(M, N, K, name, hidden):
    run_dgrad(M, N, K, name, hidden=hidden)


@pytest.mark.parametrize("M,N,K", [(20, 136, 520), (300, 200, 264)])
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4)])
def test_dgrad_pitches_and_alignment(M, N, K, pad, offset):
    run_dgrad(M, N, K, "silu", pad=pad, offset=offset)


def test_dgrad_empty_sum():
    run_dgrad(70, 0, 130, "gelu")


def run_wgrad(M, N, K, bias=True, accumulate=False, pad=0, offset=0, seed=2):
    rng = np.random.default_rng(seed + 31 * M + 7 * N + K)
    dy, x = rng_half(rng, (M, N)), rng_half(rng, (M, K))
    dw0, db0 = rng_half(rng, (N, K), 8), rng.standard_normal((1, N)).astype(np.float32)
    DY, X = Matrix(M, N, N + pad, offset, value=dy), Matrix(M, K, K + pad, offset, value=x)
    DW = Matrix(N, K, K + pad, offset, value=dw0 if accumulate else None)
    DB = Matrix(1, N, offset=offset, dtype=np.float32, value=db0 if accumulate else None) if bias else None
    tc.hgemm_linear_wgrad(DY.ptr, DY.ld, X.ptr, X.ld, DW.ptr, DW.ld, DB.ptr if DB else None, accumulate, M, N, K)
    done()
    dw, edw = ref.product(dy.T, x)
    db, edb = ref.column_sums(dy)
    if accumulate:
        dw, db = dw + dw0.astype(np.float64), db + db0[0].astype(np.float64)
        edw, edb = edw + 2.0 ** -23 * np.abs(dw), edb + 2.0 ** -23 * np.abs(db)
    what = f"wgrad {M}x{N}x{K} accumulate {accumulate} pad {pad} offset {offset}"
    check(DW.get(), dw, edw + ref.half_rounding(dw) * 1.001, what)
    if DB:
        check(DB.get()[0], db, edb + 2.0 ** -23 * np.abs(db), what + " bias")


@pytest.mark.parametrize("M,N,K", SHAPES + [(5000, 64, 128), (4100, 24, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad_shapes(M, N, K, accumulate):
    run_wgrad(M, N, K, accumulate=accumulate)


@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4)])
def test_wgrad_pitches_and_alignment(pad, offset):
    run_wgrad(300, 200, 264, pad=pad, offset=offset)
    run_wgrad(301, 136, 77, bias=False, pad=pad, offset=offset)


def test_wgrad_of_no_rows():
    run_wgrad(0, 70, 130)
    run_wgrad(0, 70, 130, accumulate=True)


def run_layernorm(M, D, pad=0, offset=0, res=True, shift=0.0, scale=1.0, eps=1e-5, in_place=None, seed=3):
    rng = np.random.default_rng(seed + 31 * M + D)
    x = (rng.standard_normal((M, D)) * scale + shift).astype(np.float16)
    gamma, beta = (1 + 0.2 * rng.standard_normal((1, D))).astype(np.float16), rng_half(rng, (1, D))
    G, B = Matrix(1, D, offset=offset, value=gamma), Matrix(1, D, offset=offset, value=beta)
    X = Matrix(M, D, D + pad, offset, value=x)
    Y = X if in_place == "x" else Matrix(M, D, D + pad, offset)
    MU, RS = Matrix(1, M, dtype=np.float32), Matrix(1, M, dtype=np.float32)
    tc.hgemm_layernorm_forward(X.ptr, X.ld, G.ptr, B.ptr, eps, Y.ptr, Y.ld, MU.ptr, RS.ptr, M, D)
    done()
    y, ey, mu, emu, rs, ers = ref.layernorm(x, gamma[0], beta[0], eps)
    what = f"layernorm {M}x{D} pad {pad} offset {offset}"
    check(Y.get(), y, ey, what)
    mean, rstd = MU.get()[0], RS.get()[0]
    check(mean, mu, emu, what + " mean")
    check(rstd, rs, ers, what + " rstd")

    X = Matrix(M, D, D + pad, offset, value=x)
    dy = rng_half(rng, (M, D), 0.5)
    r = rng_half(rng, (M, D)) if res else None
    MU, RS = Matrix(1, M, dtype=np.float32, value=mean), Matrix(1, M, dtype=np.float32, value=rstd)
    DY = Matrix(M, D, D + pad, offset, value=dy)
    R = Matrix(M, D, D + pad, offset, value=r) if res else None
    DX = DY if in_place == "dy" else R if in_place == "r" else Matrix(M, D, D + pad, offset)
    DG, DB = Matrix(1, D, offset=offset, dtype=np.float32), Matrix(1, D, offset=offset, dtype=np.float32)
    torch = torch_cuda()
    size = tc.hgemm_layernorm_backward_workspace_size(M, D)
    ws = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    tc.hgemm_layernorm_backward(DY.ptr, DY.ld, X.ptr, X.ld, G.ptr, MU.ptr, RS.ptr, R.ptr if R else None,
                                R.ld if R else 0, DX.ptr, DX.ld, DG.ptr, DB.ptr, ws, M, D, workspace_bytes=size)
    done()
    assert (ws[size:] == 0x5A).all(), "written past the workspace"
    dx, edx, dg, edg, db, edb = ref.layernorm_backward(dy, x, gamma[0], mean, rstd, r)
    check(DX.get(), dx, edx, what + " dx")
    check(DG.get()[0], dg, edg, what + " dgamma")
    check(DB.get()[0], db, edb, what + " dbeta")


@pytest.mark.parametrize("M,D", [(1, 1), (1, 4096), (2, 7), (3, 64), (1, 8200), (5, 1000), (333, 77), (64, 1024),
                                 (1000, 1000), (257, 2056), (700, 4096), (40, 8192), (3, 16384), (9, 20000),
                                 (2, 40001), (5000, 8), (4099, 72)])
def test_layernorm_shapes(M, D):
    run_layernorm(M, D, res=M % 2 == 1)


@pytest.mark.parametrize("M,D", [(70, 264), (33, 2048)])
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4)])
def test_layernorm_pitches_and_alignment(M, D, pad, offset):
    run_layernorm(M, D, pad=pad, offset=offset)


@pytest.mark.parametrize("in_place", ["x", "dy", "r"])
@pytest.mark.parametrize("M,D", [(50, 1024), (300, 200), (7, 8192), (20, 333), (3, 20000)])
def test_layernorm_in_place(M, D, in_place):
    run_layernorm(M, D, in_place=in_place)


@pytest.mark.parametrize("D", [512, 1000])
def test_layernorm_shifted_and_constant_rows(D):
    """A mean far from zero (the variance is that around the mean), and rows without variance."""
    run_layernorm(20, D, shift=100.0)
    run_layernorm(20, D, scale=0.0, shift=3.0)
    run_layernorm(20, D, scale=1e-3, eps=1e-12)


def test_layernorm_of_no_rows():
    torch = torch_cuda()
    dg, db = torch.full((72,), 5.0, device="cuda"), torch.full((72,), 5.0, device="cuda")
    g = torch.ones(72, device="cuda", dtype=torch.float16)
    ws = torch.empty(max(16, tc.hgemm_layernorm_backward_workspace_size(0, 72)), dtype=torch.uint8, device="cuda")
    tc.hgemm_layernorm_backward(None, 72, None, 72, g, None, None, None, 0, None, 72, dg, db, ws, 0, 72)
    done()
    assert (dg == 0).all() and (db == 0).all()


def run_ckpt8(x, pad=0, offset=0, name="none"):
    M, N = x.shape
    X = Matrix(M, N, N + pad, offset, value=x)
    groups = -(-N // 64)
    Q, S = Matrix(M, N, N + pad, offset, np.int8), Matrix(groups, M, M + pad, offset, np.float32)
    tc.hgemm_ckpt8_save(X.ptr, X.ld, Q.ptr, Q.ld, S.ptr, S.ld, M, N)
    Y = Matrix(M, N, N + pad, offset)
    tc.hgemm_ckpt8_load(Q.ptr, Q.ld, S.ptr, S.ld, ref.ACTS.index(name), Y.ptr, Y.ld, M, N)
    done()
    codes, scales = ref.keep32(x.astype(np.float32))
    what = f"ckpt8 {M}x{N} pad {pad} offset {offset}"
    got = Q.get()
    assert np.array_equal(got, codes), f"{what}: {np.argwhere(got != codes)[0]}"
    assert np.array_equal(S.get().view(np.uint32) & 0x7F800000, scales.view(np.uint32) & 0x7F800000), what
    check(S.get(), scales.astype(np.float64), 0.0, what + " scales")
    u = ref.kept(codes, scales)
    y = ref.act(u, name)
    check(Y.get(), y, ref.act_error(y) + 2.0 ** -23 * np.abs(u) + ref.half_rounding(y) * 1.001, what + " load")


@pytest.mark.parametrize("M,N", [(1, 1), (1, 64), (3, 65), (257, 1000), (33, 63), (100, 4096), (2000, 8), (5, 20001),
                                 (300, 264)])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_ckpt8_shapes(M, N, name):
    rng = np.random.default_rng(M * 1000 + N)
    run_ckpt8(rng_half(rng, (M, N), 3), name=name)


@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (3, 0), (1, 1), (0, 1), (8, 4), (64, 16)])
def test_ckpt8_pitches_and_alignment(pad, offset):
    run_ckpt8(rng_half(np.random.default_rng(9), (70, 328), 0.1), pad=pad, offset=offset, name="silu")


def test_ckpt8_exceptions():
    """Zeros, the smallest and largest numbers, ties, infinities and NaN."""
    x = np.zeros((6, 200), np.float16)
    x[1, :64] = np.linspace(-127, 127, 64)
    x[1, 64:128] = 2.0 ** -24
    x[1, 130] = 65504
    x[2, 5] = np.inf
    x[3, 70] = np.nan
    x[4, 190] = -np.inf
    x[5] = (np.arange(200) % 128 - 63.5)  # half steps of a scale of 0.5
    run_ckpt8(x)


def test_poisoned_groups_reach_the_gradient():
    """A NaN scale makes the whole group's dU and H NaN, and nothing else."""
    torch = torch_cuda()
    M, N, K = 130, 64, 200
    rng = np.random.default_rng(5)
    codes, scales = ref.keep32(rng.standard_normal((M, K)).astype(np.float32))
    scales[1, 7] = np.nan
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    dy, w = dev(rng_half(rng, (M, N))), dev(rng_half(rng, (N, K)))
    du, h = (torch.empty((M, K), dtype=torch.float16, device="cuda") for _ in range(2))
    for name in ref.ACTS:
        tc.hgemm_linear_dgrad(dy, N, w, K, dev(codes), K, dev(scales), M, ref.ACTS.index(name), du, K, h, K, M, N, K)
        done()
        want = np.zeros((M, K), bool)
        want[7, 64:128] = True
        assert np.array_equal(np.isnan(du.cpu().numpy()), want) or name == "none", name
        assert np.array_equal(np.isnan(h.cpu().numpy()), want), name


def test_gradients_are_differences_of_the_kernels():
    """L = Σ dY ⊙ (f(U)·Wᵀ): the kernels' dU against central differences of
    the 64-bit loss at the values the 8-bit form stands for."""
    torch = torch_cuda()
    M, N, K = 5, 24, 136
    rng = np.random.default_rng(6)
    codes, scales = ref.keep32((rng.standard_normal((M, K)) * 2).astype(np.float32))
    dy, w = rng_half(rng, (M, N)), rng_half(rng, (N, K), 0.2)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    du, h = (torch.empty((M, K), dtype=torch.float16, device="cuda") for _ in range(2))
    u = ref.kept(codes, scales)
    for name in ("gelu", "silu", "gelu_erf"):
        tc.hgemm_linear_dgrad(dev(dy), N, dev(w), K, dev(codes), K, dev(scales), M, ref.ACTS.index(name), du, K, h, K,
                              M, N, K)
        done()
        step = 1e-4
        g = dy.astype(np.float64) @ w.astype(np.float64)
        want = g * (ref.act(u + step, name) - ref.act(u - step, name)) / (2 * step)
        _, bound, _, _ = ref.dgrad(dy, w, codes, scales, name)
        check(du.cpu().numpy(), want, bound + 1e-7 * np.abs(g), f"differences {name}")


def test_equal_calls_give_equal_bits_and_follow_their_stream():
    """On a stream that is busy, with the operands written just before on it."""
    torch = torch_cuda()
    M, N, K = 500, 1000, 520
    rng = np.random.default_rng(8)
    src = {k: torch.from_numpy(v).cuda() for k, v in
           {"x": rng_half(rng, (M, K)), "w": rng_half(rng, (N, K)), "dy": rng_half(rng, (M, N))}.items()}
    side = torch.cuda.Stream()
    results = []
    for _ in range(3):
        x, w, dy = (torch.zeros_like(src[k]) for k in ("x", "w", "dy"))
        y, dw = torch.empty((M, N), **(f16 := dict(dtype=torch.float16, device="cuda"))), torch.empty((N, K), **f16)
        q = torch.empty((M, N), dtype=torch.int8, device="cuda")
        s = torch.empty((16, M), device="cuda")
        db = torch.empty(N, device="cuda")
        du, u = torch.empty((M, K), **f16), torch.empty((M, N), **f16)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy = torch.randn(4096, 4096, device="cuda")
            for _ in range(3):
                busy = busy @ busy * 1e-3
            for a, k in ((x, "x"), (w, "w"), (dy, "dy")):
                a.copy_(src[k], non_blocking=True)
            tc.hgemm_linear(x, K, w, K, None, tc.HGEMM_ACT_GELU, None, 0, y, N, M, N, K, q, N, s, M)
            tc.hgemm_ckpt8_load(q, N, s, M, tc.HGEMM_ACT_NONE, u, N, M, N)
            tc.hgemm_linear_dgrad(dy, N, w, K, None, 0, None, 0, 0, du, K, None, 0, M, N, K)
            tc.hgemm_linear_wgrad(dy, N, x, K, dw, K, db, False, M, N, K)
        assert tc.hgemm_device_status(side) == tc.HGEMM_OK
        results.append([t.cpu() for t in (y, q, s, u, du, dw, db)])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
    y, _, _, _ = ref.linear(src["x"].cpu().numpy(), src["w"].cpu().numpy(), None, "gelu", None)
    assert np.abs(results[0][0].numpy() - y).max() < 0.1


PATHS = {"narrow": tc.HGEMM_PATH_TC_NARROW, "tile": tc.HGEMM_PATH_TC, "pair": tc.HGEMM_PATH_TC_PAIR,
         "wide": tc.HGEMM_PATH_TC_WIDE, "split": tc.HGEMM_PATH_SKINNY, "any": tc.HGEMM_PATH_GENERIC}


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M,N,K", [(300, 264, 520), (20, 1000, 1000), (700, 520, 1100)])
def test_every_kernel_has_the_epilogues(path, M, N, K):
    """The same products on each product kernel (a forced path that cannot
    take one leaves it to another)."""
    tc.hgemm_force_path(PATHS[path])
    try:
        run_linear(M, N, K, "gelu", keep=True)
        run_linear(M, N, K, "silu", in_place=True)
        run_dgrad(M, N, K, "gelu")
        run_dgrad(M, N, K, None)
        run_wgrad(M, N, K, accumulate=True)
    finally:
        tc.hgemm_force_path(-1)


@pytest.mark.parametrize("M,N,K", [(9, 2048, 1024), (16, 1032, 2048), (40, 2051, 1000), (64, 264, 4096),
                                   (100, 520, 4104), (128, 9800, 264)])
def test_few_rows(M, N, K):
    run_linear(M, N, K, "gelu_erf")
    run_linear(M, N, K, "none", bias=False, in_place=True)
    run_dgrad(M, K, N, "silu")
    run_dgrad(M, K, N, None)


@pytest.mark.parametrize("M,N,K", [(129, 264, 136), (300, 72, 520), (257, 1032, 1000), (1000, 520, 1100), (640, 8, 64),
                                   (384, 328, 4104)])
def test_one_wave_of_clusters(M, N, K):
    """Odd numbers of 128×64 tiles either way, outputs that end inside one,
    contractions shorter and longer than the ring."""
    run_linear(M, N, K, "silu", keep=True)
    run_linear(M, N, K, "gelu", in_place=True)
    run_dgrad(M, K, N, "gelu")
    run_dgrad(M, K, N, None)
    run_wgrad(K, M, N, accumulate=True)
    run_wgrad(K, M, N, bias=False)


@pytest.mark.parametrize("M,N,K", [(200, 131, 3001), (150, 257, 2049), (300, 129, 1024), (200, 131, 1536)])
def test_odd_sizes_of_few_tiles_and_a_long_contraction(M, N, K):
    run_linear(M, N, K, "gelu", keep=True)
    run_linear(M, N, K, "none", in_place=True)
    run_dgrad(M, K, N, "silu")
    run_wgrad(K, N, M, accumulate=True)
    run_wgrad(K, M, N, pad=3)


@pytest.mark.parametrize("M,N,K", [(2048, 264, 136), (5000, 72, 520), (3000, 130, 128)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_small_weights_of_many_rows(M, N, K, accumulate):
    run_wgrad(M, N, K, accumulate=accumulate)
    run_wgrad(M, N, K, bias=False, accumulate=accumulate)


@pytest.mark.parametrize("M,N,K", [(300, 4360, 2056), (2050, 2600, 2048), (77, 9000, 1032)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_bias_gradient_beside_many_tiles(M, N, K, accumulate):
    run_wgrad(M, N, K, accumulate=accumulate)


def test_bias_gradient_beside_its_product():
    """The column sums may run beside the product: what comes before the pair
    of launches on the stream and what comes after keep their order."""
    torch = torch_cuda()
    M, N, K = 4096, 1024, 2048
    rng = np.random.default_rng(12)
    src = torch.from_numpy(rng_half(rng, (M, N))).cuda()
    x = torch.from_numpy(rng_half(rng, (M, K))).cuda()
    dy, dw, db = torch.empty_like(src), torch.empty((N, K), dtype=torch.float16, device="cuda"), torch.empty(N, device="cuda")
    want = src.double().sum(dim=0)
    first = None
    for _ in range(20):
        dy.fill_(float("nan"))
        dw.fill_(float("nan"))
        db.fill_(float("nan"))
        dy.copy_(src)
        tc.hgemm_linear_wgrad(dy, N, x, K, dw, K, db, False, M, N, K)
        copies = dw.clone(), db.clone()
        dy.zero_()
        tc.hgemm_linear_wgrad(dy, N, x, K, dw, K, db, True, M, N, K)   # adds nothing
        dy.fill_(1.0)
        assert torch.equal(dw, copies[0]) and torch.equal(db, copies[1])
        assert (copies[1].double() - want).abs().max() < 1e-3 * want.abs().max()
        first = first or copies
        assert torch.equal(first[0], copies[0]) and torch.equal(first[1], copies[1])
    done()


@pytest.mark.parametrize("what", ["pair", "narrow", "split", "few rows", "few rows back", "small weight", "clusters",
                                  "any", "any shared", "norm"])
def test_withheld_arrival_times_out(what):
    """Each kernel's waits are bounded: a withheld arrival ends in a timeout
    the host reads, and the context computes on."""
    torch = torch_cuda()
    half = lambda *s: torch.ones(s, dtype=torch.float16, device="cuda")  # noqa: E731
    y, w = half(2048, 512), half(512, 512)
    db, ws = torch.empty(512, device="cuda"), torch.empty(tc.hgemm_layernorm_backward_workspace_size(64, 512),
                                                        dtype=torch.uint8, device="cuda")
    stats = torch.ones(64, device="cuda")
    calls = {
        "pair": lambda: tc.hgemm_linear(y, 512, w, 512, None, 2, None, 0, half(600, 512), 512, 600, 512, 512),
        "few rows": lambda: tc.hgemm_linear(y, 512, half(8192, 512), 512, None, 2, None, 0, half(40, 8192), 8192, 40,
                                            8192, 512),
        "few rows back": lambda: tc.hgemm_linear_dgrad(y, 512, w, 512, None, 0, None, 0, 0, half(20, 512), 512, None, 0,
                                                       20, 512, 512),
        "small weight": lambda: tc.hgemm_linear_wgrad(y, 512, y, 512, half(512, 512), 512, None, False, 2048, 512, 512),
        "clusters": lambda: tc.hgemm_linear_dgrad(y, 512, w, 512, None, 0, None, 0, 0, half(600, 512), 512, None, 0, 600,
                                                  512, 512),
        "any": lambda: tc.hgemm_linear(y, 511, w, 511, None, 2, None, 0, half(600, 512), 511, 600, 511, 511),
        "any shared": lambda: tc.hgemm_linear(half(200, 2049), 2049, half(199, 2049), 2049, None, 2, None, 0, half(200, 199),
                                              199, 200, 199, 2049),
        "norm": lambda: tc.hgemm_layernorm_backward(y, 512, y, 512, w, stats, stats, None, 0, half(64, 512), 512, db,
                                                    torch.empty(512, device="cuda"), ws, 64, 512),
    }
    calls["narrow"] = calls["split"] = calls["pair"]
    done()
    tc.hgemm_set_wait_timeout(20_000_000)
    tc.hgemm_debug_inject(tc.HGEMM_INJECT_DROP_ARRIVAL)
    if what in ("pair", "narrow", "split"):
        tc.hgemm_force_path(PATHS[what])
    try:
        calls[what]()
        assert tc.hgemm_device_status() == tc.HGEMM_ERR_TIMEOUT
        assert tc.hgemm_device_status() == tc.HGEMM_OK
    finally:
        tc.hgemm_debug_inject(tc.HGEMM_INJECT_NONE)
        tc.hgemm_set_wait_timeout(0)
        tc.hgemm_force_path(-1)
    run_linear(300, 264, 520, "gelu", keep=True)
    run_layernorm(40, 512)
