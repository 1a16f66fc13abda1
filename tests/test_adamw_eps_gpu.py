"""AdamW's eps at its smallest: a value without a gradient stays (GPU only)."""

import numpy as np
import pytest

import tensor_core_dense_fp16_gb300 as tc
from test_adamw_gpu import Array, table
from test_block_gpu import done

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [1e-30, 2.0 ** -126, 1e-40, 1e-45, 1e-60, 5e-324])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("n", [4096, 77])
def test_values_without_a_gradient(eps, bits, n):
    rng = np.random.default_rng(n)
    g, p = np.zeros(n, np.float32), rng.standard_normal(n).astype(np.float32)
    g[::3] = 0.5
    t = {"grad": g, "master": p, "m": np.zeros(n, np.int8 if bits == 8 else np.float32),
         "v": np.zeros(n, np.uint8 if bits == 8 else np.float32)}
    if bits == 8:
        t["m_scales"], t["v_scales"] = (np.zeros(-(-n // 64), np.float32) for _ in range(2))
    t = {k: Array(a) for k, a in t.items()}
    tc.hgemm_adamw(table([(t, 0.0)]), 1e-2, eps=eps, step=1)
    done()
    got = t["master"].get()
    still = g == 0
    assert (got[still] == p[still]).all()
    # a first step is lr, within an FP32 root, reciprocal and sum
    assert (np.abs(got[~still] - (p[~still].astype(np.float64) - 1e-2)) <= 1e-2 * 2.0 ** -18 + 2.0 ** -23 * np.abs(p[~still])).all()


def test_eps_0_is_the_formulas():
    """0/0 where there has been no gradient."""
    n = 128
    t = {"grad": np.zeros(n, np.float32), "master": np.ones(n, np.float32), "m": np.zeros(n, np.float32),
         "v": np.zeros(n, np.float32)}
    t["grad"][1] = 1
    t = {k: Array(a) for k, a in t.items()}
    tc.hgemm_adamw(table([(t, 0.0)]), 1e-2, eps=0.0, step=1)
    done()
    got = t["master"].get()
    assert np.isfinite(got[1]) and np.isnan(np.delete(got, 1)).all()
