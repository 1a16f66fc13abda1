"""Tables of tensors made from addresses (CPU: addresses are made up, no
computing call is made)."""

import pytest

import tensor_core_dense_fp16_gb300 as tc
from tensor_core_dense_fp16_gb300 import build as tcbuild
from test_around_host import A, adamw_tensor, table

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    tcbuild.build()
    return tc.load()


class Gradient:
    """What a table looks at of a tensor."""

    def __init__(self, at, n=128, dtype=torch.float16, device=0):
        self.at, self.n, self.dtype, self.index = at, n, dtype, device
        self.is_cuda, self.device, self.shape = device >= 0, f"cuda:{device}" if device >= 0 else "cpu", (n,)

    def get_device(self):
        return self.index

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


OTHER = dict(weight=A[10], master=A[11], grad=A[12], m=A[13], v=A[14])


@pytest.mark.parametrize("known", [None, 0])
def test_gradients_of_a_table_made_from_addresses(known):
    plan = tc.AdamwTensors(table(adamw_tensor(), adamw_tensor(**OTHER)), [], device=known)
    good = [Gradient(A[15]), Gradient(A[16], dtype=torch.float32)]
    plan.set_gradients(good)
    assert [(r.grad, r.grad_type) for r in plan.table] == [(A[15], tc.HGEMM_TYPE_F16), (A[16], tc.HGEMM_TYPE_F32)]
    assert plan.grads == good
    before = bytes(plan.table)
    for bad in (Gradient(A[17], device=-1), Gradient(A[17], device=1), Gradient(A[17], n=127)):
        with pytest.raises(ValueError):
            plan.set_gradients([good[0], bad])
    with pytest.raises(ValueError):
        plan.set_gradients([Gradient(A[17], device=-1), good[1]])
    with pytest.raises(TypeError):
        plan.set_gradients([good[0], Gradient(A[17], dtype=torch.float64)])
    with pytest.raises(tc.HgemmError):
        plan.set_gradients([good[0], Gradient(A[3])])
    assert bytes(plan.table) == before and plan.grads == good
