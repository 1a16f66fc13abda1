"""The experts' workspace of a largest batch serves every smaller one (CPU: sizes
and checks of arguments; no computing call is made)."""

import pytest

import tensor_core_dense_fp16_gb300 as tc
from tensor_core_dense_fp16_gb300 import build as tcbuild

# narrow layers, whose F is cut into the more runs the fewer experts are chosen
NARROW = [(256, 1024, 64, 1), (128, 1024, 128, 2), (64, 4096, 512, 4), (200, 2048, 100, 1)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    tcbuild.build()
    return tc.load()


@pytest.mark.parametrize("d,f,e,k", NARROW + [(d, f, e, k) for d in (1, 40, 512, 4096) for f in (0, 77, 512, 8192)
                                              for e in (1, 8, 64, 512) for k in (1, 2, 16) if k <= e])
def test_the_size_does_not_fall_with_more_tokens(d, f, e, k):
    sizes = [tc.hgemm_experts_workspace_size(m, d, f, e, k) for m in range(65)]
    assert sizes == sorted(sizes)
