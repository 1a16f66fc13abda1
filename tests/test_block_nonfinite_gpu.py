"""Infinities and NaN through the block's operators: they reach what the
formulas say, on every kernel, and nothing else (GPU only)."""

import numpy as np
import pytest

import block_reference as ref
import tensor_core_dense_fp16_gb300 as tc
from gpu_helpers import torch_cuda
from test_block_gpu import PATHS

pytestmark = pytest.mark.gpu

BAD = (np.inf, -np.inf, np.nan)


def dev(a):
    return torch_cuda().from_numpy(np.ascontiguousarray(a)).cuda()


def out(*shape, dtype="float16"):
    torch = torch_cuda()
    return torch.full(shape, 77.0, dtype=getattr(torch, dtype), device="cuda")


def same_kind(got, want, bound, what):
    """NaN where the formula has NaN, its infinities, and its values within the
    bound (a value that FP16 cannot hold is infinite too)."""
    got = got.cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        want16 = np.where(np.abs(want) >= 65520, np.copysign(np.inf, want), want)
        near = np.abs(np.abs(want) - 65520) < 64
        ok = np.where(np.isnan(want), np.isnan(got), np.where(np.isinf(want16), got == want16, np.abs(got - want) <= bound))
    assert (ok | near).all(), (what, np.argwhere(~ok)[:4], got[~ok][:4], want[~ok][:4])


def products(a, b):
    """a·b in 64 bits with IEEE infinities and NaN, and a bound where it is finite."""
    with np.errstate(invalid="ignore", over="ignore"):
        u = a.astype(np.float64) @ b.astype(np.float64)
    _, bound = ref.product(np.nan_to_num(a, nan=0, posinf=0, neginf=0), np.nan_to_num(b, nan=0, posinf=0, neginf=0))
    return u, bound


def sprinkle(rng, a, rows):
    """One bad value in each of some rows: the first, the last and some other place."""
    a = a.copy()
    for i, r in enumerate(rows):
        c = (0, a.shape[1] - 1, int(rng.integers(a.shape[1])))[i // 3 % 3]
        a[r, c] = BAD[i % 3]
    return a


# one row, few rows, a batch, one wave, more tiles, split K, odd sizes, odd outputs alone
SHAPES = [(1, 264, 520), (7, 65, 77), (24, 1032, 136), (100, 520, 2056), (300, 264, 200), (2100, 2048, 136),
          (200, 136, 8200), (150, 131, 71), (300, 129, 136)]


def rows_of(m):
    return sorted({0, m - 1, m // 2, m // 3, m // 5, 2 * m // 3})


def check_linear(M, N, K, name, keep):
    rng = np.random.default_rng(M + N + K)
    x = sprinkle(rng, rng.standard_normal((M, K)).astype(np.float16), rows_of(M))
    w = (rng.standard_normal((N, K)) / K ** 0.5).astype(np.float16)
    w[N // 2, K // 2] = np.nan
    w[0, K - 1] = np.inf
    y, q, s, back = out(M, N), out(M, N, dtype="int8"), out(-(-N // 64), M, dtype="float32"), out(M, N)
    tc.hgemm_linear(dev(x), K, dev(w), K, None, ref.ACTS.index(name), None, 0, y, N, M, N, K, q if keep else None, N,
                    s if keep else None, M)
    if keep:
        tc.hgemm_ckpt8_load(q, N, s, M, 0, back, N, M, N)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    u, eu = products(x, w.T)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.act(u, name)
        bound = ref.LIPSCHITZ * eu + ref.act_error(want) + ref.half_rounding(want) * 1.001
    same_kind(y, want, bound, f"linear {M}x{N}x{K} {name}")
    if keep:
        # a group that holds an infinity or a NaN reads back as NaN, and only it
        groups = -(-N // 64)
        padded = np.zeros((M, groups * 64))
        padded[:, :N] = u
        bad = ~np.isfinite(padded.reshape(M, groups, 64)).all(axis=2)
        assert np.array_equal(np.isnan(s.cpu().numpy().T), bad)
        assert np.array_equal(np.isnan(back.cpu().numpy()), np.repeat(bad, 64, axis=1)[:, :N])
        assert not q.cpu().numpy()[np.repeat(bad, 64, axis=1)[:, :N]].any()


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("name", ref.ACTS)
def test_linear(M, N, K, name):
    check_linear(M, N, K, name, False)
    check_linear(M, N, K, name, True)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_input_gradient(M, N, K):
    rng = np.random.default_rng(M + N + K)
    dy = sprinkle(rng, rng.standard_normal((M, N)).astype(np.float16), rows_of(M))
    w = (rng.standard_normal((N, K)) / N ** 0.5).astype(np.float16)
    w[N - 1, K // 3] = -np.inf
    codes, scales = ref.keep32(rng.standard_normal((M, K)).astype(np.float32))
    du, plain = out(M, K), out(M, K)
    tc.hgemm_linear_dgrad(dev(dy), N, dev(w), K, None, 0, None, 0, 0, plain, K, None, 0, M, N, K)
    tc.hgemm_linear_dgrad(dev(dy), N, dev(w), K, dev(codes), K, dev(scales), M, tc.HGEMM_ACT_SILU, du, K, None, 0, M, N,
                          K)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    g, eg = products(dy, w)
    with np.errstate(invalid="ignore", over="ignore"):
        same_kind(plain, g, eg + ref.half_rounding(g) * 1.001, "no activation")
        want = g * ref.act_gradient(ref.kept(codes, scales), "silu")
        same_kind(du, want, ref.LIPSCHITZ * eg + 2.0 ** -18 * np.abs(g) + ref.half_rounding(want) * 1.001, "silu")


@pytest.mark.parametrize("N,K,M", SHAPES + [(128, 136, 8200)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient(M, N, K, accumulate):
    rng = np.random.default_rng(M + N + K)
    dy = rng.standard_normal((M, N)).astype(np.float16)
    x = rng.standard_normal((M, K)).astype(np.float16)
    dy.T[:] = sprinkle(rng, dy.T, rows_of(N))
    x[M - 1, K // 2], x[0, 0] = np.inf, np.nan
    dw, db = out(N, K), out(N, dtype="float32")
    tc.hgemm_linear_wgrad(dev(dy), N, dev(x), K, dw, K, db, accumulate, M, N, K)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    want, bound = products(dy.T, x)
    with np.errstate(invalid="ignore", over="ignore"):
        sums = dy.astype(np.float64).sum(axis=0)
    _, eb = ref.column_sums(np.nan_to_num(dy, nan=0, posinf=0, neginf=0))
    old = 77.0 if accumulate else 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        want = want + old
        same_kind(dw, want, bound + 2.0 ** -23 * np.abs(want) + ref.half_rounding(want) * 1.001, "dW")
        same_kind(db, sums + old, eb + 2.0 ** -23 * np.abs(sums + old), "dbias")


@pytest.mark.parametrize("path", PATHS)
def test_each_product_kernel(path):
    tc.hgemm_force_path(PATHS[path])
    try:
        for M, N, K in ((300, 264, 200), (129, 72, 520)):
            check_linear(M, N, K, "gelu", True)
            test_input_gradient(M, N, K)
            test_weight_gradient(M, N, K, True)
    finally:
        tc.hgemm_force_path(-1)


# the ring's group sizes and the rows it does not take
@pytest.mark.parametrize("D", [264, 1024, 2048, 4096, 8192, 16384, 333, 20000])
def test_norm(D):
    M = 12
    rng = np.random.default_rng(D)
    x = sprinkle(rng, rng.standard_normal((M, D)).astype(np.float16), (1, 4, 9))
    gamma = (1 + 0.1 * rng.standard_normal(D)).astype(np.float16)
    beta = rng.standard_normal(D).astype(np.float16)
    y, mean, rstd = out(M, D), out(M, dtype="float32"), out(M, dtype="float32")
    tc.hgemm_layernorm_forward(dev(x), D, dev(gamma), dev(beta), 1e-5, y, D, mean, rstd, M, D)
    assert tc.hgemm_device_status() == tc.HGEMM_OK
    bad = np.zeros(M, bool)
    bad[[1, 4, 9]] = True
    with np.errstate(invalid="ignore"):
        want, bound, mu, emu, rs, ers = ref.layernorm(x, gamma, beta, 1e-5)
    same_kind(y, want, bound, "y")
    same_kind(mean, mu, emu, "mean")
    same_kind(rstd, rs, ers, "rstd")
    assert np.array_equal(np.isnan(y.cpu().numpy()).all(axis=1), bad)

    # backward: a bad x spoils its row and dgamma; a bad dY its row and its column of both sums
    for spoil in ("x", "dy", "r"):
        clean = rng.standard_normal((M, D)).astype(np.float16)
        dy, r = (0.1 * rng.standard_normal((2, M, D))).astype(np.float16)
        xs = x if spoil == "x" else clean
        dy = sprinkle(rng, dy, (0, 5, 11)) if spoil == "dy" else dy
        r = sprinkle(rng, r, (2, 3, 7)) if spoil == "r" else r
        with np.errstate(invalid="ignore"):
            x64 = xs.astype(np.float64)
            mu = x64.mean(axis=1).astype(np.float32)
            rs = (1 / np.sqrt(x64.var(axis=1) + 1e-5)).astype(np.float32)
        dx, dg, db = out(M, D), out(D, dtype="float32"), out(D, dtype="float32")
        ws = torch_cuda().empty(tc.hgemm_layernorm_backward_workspace_size(M, D), dtype=torch_cuda().uint8, device="cuda")
        tc.hgemm_layernorm_backward(dev(dy), D, dev(xs), D, dev(gamma), dev(mu), dev(rs), dev(r), D, dx, D, dg, db, ws, M,
                                    D)
        assert tc.hgemm_device_status() == tc.HGEMM_OK
        with np.errstate(invalid="ignore"):
            want = ref.layernorm_backward(dy, xs, gamma, mu, rs, r)
            for got, value, b, what in zip((dx, dg, db), want[::2], want[1::2], ("dx", "dgamma", "dbeta")):
                same_kind(got, value, b, f"{what}, bad {spoil}")
