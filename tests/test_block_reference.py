"""The 64-bit reference of the feed-forward block's operators against
differences of its own forward formulas, and hand values (CPU)."""

import numpy as np
import pytest

import block_reference as ref


@pytest.mark.parametrize("name", ref.ACTS)
def test_activation_gradient_is_the_difference_quotient(name):
    u = np.linspace(-6, 6, 241) + 1e-3  # off relu's corner
    h = 1e-5
    want = (ref.act(u + h, name) - ref.act(u - h, name)) / (2 * h)
    # central difference: h²/6·|f'''| < 1e-10, cancellation 2^-52·6/h < 2e-10
    assert np.abs(ref.act_gradient(u, name) - want).max() < 1e-8


def test_activation_values():
    assert ref.act(np.array([1.0]), "silu")[0] == pytest.approx(0.7310585786300049, rel=1e-14)
    assert ref.act(np.array([1.0]), "gelu")[0] == pytest.approx(0.8411919906082768, rel=1e-14)
    assert ref.act(np.array([1.0]), "gelu_erf")[0] == pytest.approx(0.8413447460685429, rel=1e-14)


def test_layernorm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(3)
    m, d, eps = 3, 7, 1e-5
    x, dy = rng.standard_normal((m, d)), rng.standard_normal((m, d))
    gamma, beta = rng.standard_normal(d), rng.standard_normal(d)

    def loss(x, gamma, beta):
        return (dy * ref.layernorm(x, gamma, beta, eps)[0]).sum()

    _, _, mu, _, rstd, _ = ref.layernorm(x, gamma, beta, eps)
    dx, _, dgamma, _, dbeta, _ = ref.layernorm_backward(dy, x, gamma, mu, rstd, None)
    h = 1e-5
    for i in range(m):
        for j in range(d):
            e = np.zeros((m, d))
            e[i, j] = h
            assert dx[i, j] == pytest.approx((loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h), abs=1e-7)
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert dgamma[j] == pytest.approx((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h), abs=1e-7)
        assert dbeta[j] == pytest.approx((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h), abs=1e-7)


def test_dgrad_and_wgrad_are_difference_quotients():
    """L = Σ dY ⊙ (f(U)·Wᵀ): dL/dU and dL/dW."""
    rng = np.random.default_rng(4)
    m, n, k = 3, 5, 70
    codes = rng.integers(-127, 128, size=(m, k)).astype(np.int8)
    scales = rng.uniform(0.005, 0.02, size=(2, m)).astype(np.float32)
    u = ref.kept(codes, scales)
    w, dy = rng.standard_normal((n, k)), rng.standard_normal((m, n))
    h = 1e-5
    for name in ref.ACTS:
        du, _, hid, _ = ref.dgrad(dy, w, codes, scales, name)
        for i, j in ((0, 0), (1, 63), (2, 64), (2, 69)):
            if name == "relu" and abs(u[i, j]) < 2 * h:
                continue
            e = np.zeros((m, k))
            e[i, j] = h
            want = ((dy * (ref.act(u + e, name) @ w.T)).sum() - (dy * (ref.act(u - e, name) @ w.T)).sum()) / (2 * h)
            assert du[i, j] == pytest.approx(want, abs=1e-7)
        dw = ref.product(dy.T, hid)[0]
        e = np.zeros((n, k))
        e[4, 65] = h
        want = ((dy * (hid @ (w + e).T)).sum() - (dy * (hid @ (w - e).T)).sum()) / (2 * h)
        assert dw[4, 65] == pytest.approx(want, abs=1e-7)


def test_eight_bit_form():
    x = np.zeros((4, 130), np.float32)
    x[0, :64] = np.linspace(-127, 127, 64)
    x[1, 3] = np.inf
    x[2, 70] = np.nan
    x[3, 128] = -2.0
    codes, scales = ref.keep32(x)
    assert scales.shape == (3, 4) and codes.shape == (4, 130)
    assert scales[0, 0] == 1 and codes[0, 0] == -127 and codes[0, 63] == 127
    assert np.isnan(scales[0, 1]) and (codes[1] == 0).all() and scales[1, 1] == 0
    assert np.isnan(scales[1, 2]) and scales[0, 2] == 0
    assert codes[3, 128] == -127 and scales[2, 3] == np.float32(2) / np.float32(127)
