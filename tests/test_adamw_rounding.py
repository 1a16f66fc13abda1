"""The choice of a rounding: its checks of arguments (CPU; no computing call is
made, addresses are made up) and the reference's random numbers."""

import numpy as np
import pytest

import rounding_reference as rounded
import tensor_core_dense_fp16_gb300 as tc
from tensor_core_dense_fp16_gb300 import build as tcbuild
from test_around_host import ALIAS, BAD, OK, A, adamw_tensor, table


@pytest.fixture(scope="module")
def lib():
    tcbuild.build()
    return tc.load()


def test_refusals(lib):
    def call(t, rounding, lr=1e-3, step=1):
        return lib.hgemm_adamw_rounded(t, len(t), lr, 0.9, 0.999, 1e-8, step, 1.0, rounding, None, None)

    empty = table(adamw_tensor(n=0, weight=None, master=None, grad=None, m=None, v=None))
    for rounding in (tc.HGEMM_ROUND_NEAREST, tc.HGEMM_ROUND_RANDOM):
        assert call(empty, rounding) == OK
        assert call(empty, rounding, step=0) == BAD and call(empty, rounding, lr=float("nan")) == BAD
        assert call(table(adamw_tensor(m=A[0])), rounding) == ALIAS
        assert call(table(adamw_tensor(grad=None)), rounding) == BAD
    for rounding in (-1, 2):
        assert call(empty, rounding) == BAD
    with pytest.raises(tc.HgemmError):
        tc.hgemm_adamw_rounded(tc.AdamwTensors(table(), []), 1e-3, stream=0, rounding=2)


def test_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(tcbuild.INCLUDE, "hgemm.h"), encoding="utf-8").read()
    found = dict(re.findall(r"#define\s+(HGEMM_ROUND_\w+)\s+(\d+)", text))
    assert found == {n: str(getattr(tc, n)) for n in ("HGEMM_ROUND_NEAREST", "HGEMM_ROUND_RANDOM")}


def test_the_reference_rounds_to_the_value_in_the_mean():
    """Over 4000 steps of the same values: a code's value in the mean, within six
    deviations of half a step (the largest) over √4000."""
    rng = np.random.default_rng(0)
    m = rng.standard_normal(128).astype(np.float32)
    v = np.square(rng.standard_normal(128)).astype(np.float32)
    steps = range(1, 4001)
    sums = np.zeros((2, 128))
    for step in steps:
        codes, scales = rounded.keep_m(m, step)
        sums[0] += codes * np.repeat(scales, 64).astype(np.float64)
        codes, scales = rounded.keep_v(v, step)
        c = codes.astype(np.int64) - 255
        sums[1] += np.where(codes > 0, 2.0 ** (c // 8) * (1 + c % 8 / 8), 0) * np.repeat(scales, 64)
    mean = sums / len(steps)
    step_m = np.repeat(np.abs(m).reshape(2, 64).max(axis=1) / 127, 64)
    assert (np.abs(mean[0] - m) < step_m * (3 / 4000 ** 0.5 + 2.0 ** -12)).all()
    assert (np.abs(mean[1] - v) < v / 8 * (3 / 4000 ** 0.5 + 2.0 ** -12)).all()
