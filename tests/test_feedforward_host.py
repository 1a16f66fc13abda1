"""Argument checks of the feed-forward block (CPU: no computing call is made)."""

import numpy as np
import pytest

import tensor_core_dense_fp16_gb300 as tc

torch = pytest.importorskip("torch")

from tensor_core_dense_fp16_gb300.feedforward import FeedForward, Saved  # noqa: E402

D, F = 64, 136


def half(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def block():
    return FeedForward(half(D), half(D), half(F, D), half(F), half(D, F), half(D))


def saved(m):
    return dict(x=half(m, D), mean=torch.zeros(m), rstd=torch.zeros(m), codes=torch.zeros(m, F, dtype=torch.int8),
                scales=torch.zeros(3, m))


@pytest.mark.parametrize("name,value", [("x", half(4, D)), ("mean", torch.zeros(4)), ("rstd", torch.zeros(4)),
                                        ("codes", torch.zeros(5, F - 8, dtype=torch.int8)),
                                        ("scales", torch.zeros(2, 5)), ("scales", torch.zeros(5, 3).t()),
                                        ("x", half(5, 2 * D)[:, :D])])
def test_backward_refuses_what_another_forward_saved(name, value):
    with pytest.raises(ValueError, match=f"saved {name}"):
        block().backward(half(5, D), Saved(**{**saved(5), name: value}))


def test_backward_refuses_more_rows_than_were_saved():
    with pytest.raises(ValueError, match="saved x"):
        block().backward(half(6, D), Saved(**saved(5)))


def test_rows_and_weights_are_checked():
    for x in (half(D), half(4, D + 8), half(4, 2 * D)[:, :D]):
        with pytest.raises(ValueError, match="contiguous M×64"):
            block()(x)
    with pytest.raises(ValueError, match="w2 must be"):
        FeedForward(half(D), half(D), half(F, D), half(F), half(F, D), half(D))
    with pytest.raises(ValueError, match="w1 must be contiguous"):
        FeedForward(half(D), half(D), half(D, F).t(), half(F), half(D, F), half(D))
    with pytest.raises(KeyError):
        FeedForward(half(D), half(D), half(F, D), half(F), half(D, F), half(D), act="tanh")


@pytest.mark.parametrize("workspace", [torch.zeros(1 << 20, dtype=torch.uint8), np.zeros(1 << 20, np.uint8)])
def test_a_workspace_in_host_memory_is_refused(workspace):
    a = [0x10000000 * (i + 1) for i in range(10)]
    with pytest.raises(ValueError, match="workspace"):
        tc.hgemm_layernorm_backward(a[0], 64, a[1], 64, a[2], a[3], a[4], None, 0, a[5], 64, a[6], a[7], workspace, 0,
                                    64, stream=0)
