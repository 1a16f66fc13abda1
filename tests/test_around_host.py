"""Argument checks of the operators around the feed-forward block (CPU: no
computing call is made; addresses are made up)."""

import ctypes
import os
import re

import pytest

import tensor_core_dense_fp16_gb300 as tc
from tensor_core_dense_fp16_gb300 import build as tcbuild
from test_block_host import ALIAS, BAD, OK, caller

A = [0x10000000 * (i + 1) for i in range(24)]  # 16-byte aligned, disjoint


@pytest.fixture(scope="module")
def lib():
    tcbuild.build()
    return tc.load()


def test_residual_norm_forward(lib):
    names = ("X ldx alpha Y ldy gate post post_gamma post_beta pre pre_gamma pre_beta eps Z ldz H ldh stats M D").split()
    call = caller(lib.hgemm_residual_norm_forward, names,
                  dict(X=A[0], ldx=64, alpha=1.0, Y=A[1], ldy=64, gate=A[2], post=1, post_gamma=A[3], post_beta=A[4],
                       pre=2, pre_gamma=A[5], pre_beta=A[6], eps=1e-5, Z=A[7], ldz=64, H=A[8], ldh=64, stats=A[9],
                       M=16, D=64))
    for kw in (dict(M=-1), dict(D=1 << 31), dict(post=3), dict(pre=-1), dict(post=0), dict(pre=0),
               dict(post=0, post_gamma=None), dict(pre=0, pre_gamma=None, pre_beta=None), dict(post_gamma=None),
               dict(pre_gamma=None), dict(H=None), dict(X=None), dict(Y=None), dict(Z=None), dict(ldx=63),
               dict(ldy=63), dict(ldz=63), dict(ldh=63), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(alpha=float("nan")), dict(alpha=float("inf")), dict(X=A[0] + 1),
               dict(stats=A[9] + 2), dict(gate=A[2] + 1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(Z=A[0] + 2), dict(Z=A[0], ldz=72), dict(Z=A[1]), dict(H=A[0]), dict(H=A[1] + 2),
               dict(H=A[1], ldh=72), dict(Z=A[8]), dict(Z=A[3]), dict(H=A[6]), dict(stats=A[0]), dict(stats=A[7]),
               dict(stats=A[8] + 4), dict(stats=A[2])):
        assert call(**kw) == ALIAS, kw
    assert call(M=0) == OK and call(D=0) == OK
    assert call(M=0, X=None, Y=None, Z=None, H=None, stats=None) == OK


def test_residual_norm_backward(lib):
    size = tc.hgemm_residual_norm_backward_workspace_size
    need = size(16, 64)
    assert need > 0 and size(0, 0) == 0 and size(-1, 64) == 0 and size(16, 1 << 31) == 0
    assert all(size(m, d) <= 160 * 4 * (d + 32) * 4 for m in (1, 16384, 1 << 20) for d in (1, 64, 77, 8192))
    names = ("dZ lddz dH lddh Z ldz Y ldy alpha gate post post_gamma post_beta pre pre_gamma stats dX lddx dY lddy "
             "dgate dpost_gamma dpost_beta dpre_gamma dpre_beta ws bytes M D").split()
    call = caller(lib.hgemm_residual_norm_backward, names,
                  dict(dZ=A[0], lddz=64, dH=A[1], lddh=64, Z=A[2], ldz=64, Y=A[3], ldy=64, alpha=1.0, gate=A[4],
                       post=1, post_gamma=A[5], post_beta=A[6], pre=2, pre_gamma=A[7], stats=A[8], dX=A[9], lddx=64,
                       dY=A[10], lddy=64, dgate=A[11], dpost_gamma=A[12], dpost_beta=A[13], dpre_gamma=A[14],
                       dpre_beta=A[15], ws=A[16], bytes=need, M=16, D=64))
    for kw in (dict(M=-1), dict(post=4), dict(pre=3), dict(pre=0), dict(post=0), dict(dH=None), dict(Z=None),
               dict(Y=None), dict(stats=None), dict(dX=None), dict(dY=None), dict(gate=None), dict(post_gamma=None),
               dict(pre_gamma=None), dict(lddz=63), dict(lddh=63), dict(ldz=63), dict(ldy=63), dict(lddx=63),
               dict(lddy=63), dict(alpha=float("nan")), dict(ws=None), dict(ws=A[16] + 8), dict(bytes=need - 1),
               dict(dgate=A[11] + 2), dict(stats=A[8] + 2)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dX=A[1]), dict(dX=A[0], lddx=72), dict(dX=A[0] + 2), dict(dY=A[0]), dict(dY=A[1] + 2),
               dict(dX=A[2]), dict(dY=A[3]), dict(dX=A[10]), dict(dgate=A[12]), dict(dgate=A[0]), dict(dpre_beta=A[9]),
               dict(dgate=A[8]), dict(ws=A[0]), dict(ws=A[10]), dict(ws=A[15]), dict(dX=A[4]), dict(dZ=A[16])):
        assert call(**kw) == ALIAS, kw
    assert call(D=0) == OK


def adamw_tensor(**kw):
    t = tc._AdamwTensor()
    for k, v in {**dict(weight=A[0], master=A[1], grad=A[2], m=A[3], v=A[4], n=128, weight_decay=0.1, grad_type=0),
                 **kw}.items():
        setattr(t, k, v)
    return t


def table(*tensors):
    return (tc._AdamwTensor * len(tensors))(*tensors)


def test_adamw(lib):
    def call(t, count=None, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, scale=1.0, dynamic=None):
        return lib.hgemm_adamw(t, len(t) if count is None else count, lr, b1, b2, eps, step, scale, dynamic, None)

    bad = [dict(n=-1), dict(n=1 << 31), dict(grad=None), dict(m=None), dict(v=None), dict(weight=None, master=None),
           dict(grad_type=2), dict(weight_decay=float("nan")), dict(m_scales=A[5]), dict(v_scales=A[5]),
           dict(weight=A[0] + 1), dict(master=A[1] + 2), dict(m=A[3] + 1), dict(grad=A[2] + 1),
           dict(grad=A[2] + 2, grad_type=1), dict(m_scales=A[5] + 2, v_scales=A[6])]
    alias = [dict(m=A[0]), dict(v=A[3] + 4 * 127), dict(master=A[0]), dict(weight=A[2] + 2), dict(m_scales=A[4], v_scales=A[6]),
             dict(m_scales=A[5], v_scales=A[5]), dict(grad=A[1])]
    for kw in bad:
        assert call(table(adamw_tensor(**kw))) == BAD and lib.hgemm_adamw_check(table(adamw_tensor(**kw)), 1) == BAD, kw
    for kw in alias:
        t = table(adamw_tensor(**kw))
        assert call(t) == ALIAS and lib.hgemm_adamw_check(t, 1) == ALIAS, kw
    t = table(adamw_tensor(n=0, weight=None, master=None, grad=None, m=None, v=None))
    assert call(t) == OK and call(t, 0) == OK and lib.hgemm_adamw(None, 0, 1e-3, 0.9, 0.999, 1e-8, 1, 1.0, None, None) == OK
    for kw in (dict(lr=float("inf")), dict(lr=float("nan")), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0),
               dict(b2=float("nan")), dict(eps=-1e-9), dict(eps=float("inf")), dict(step=0), dict(step=-5),
               dict(scale=float("nan")), dict(count=-1), dict(dynamic=A[20] + 2)):
        assert call(t, **kw) == BAD, kw
    assert lib.hgemm_adamw(None, 1, 1e-3, 0.9, 0.999, 1e-8, 1, 1.0, None, None) == BAD
    assert call(table(adamw_tensor()), dynamic=A[3] + 8) == ALIAS

    other = dict(weight=A[10], master=A[11], grad=A[12], m=A[13], v=A[14])
    check = lib.hgemm_adamw_check
    assert check(table(adamw_tensor(), adamw_tensor(**other)), 2) == OK
    assert check(table(adamw_tensor(), adamw_tensor(**{**other, "grad": A[2]})), 2) == OK  # a shared gradient
    for name in ("weight", "master", "m", "v"):
        for victim in (A[0], A[1] + 4 * 127, A[2], A[3], A[4] + 4):
            t = table(adamw_tensor(), adamw_tensor(**{**other, name: victim}))
            assert check(t, 2) == ALIAS, (name, victim)
    assert check(table(adamw_tensor(), adamw_tensor(**{**other, "grad": A[4]})), 2) == ALIAS
    assert check(None, 0) == OK and check(None, 1) == BAD and check(None, -1) == BAD


def test_adamw_load(lib):
    call = caller(lib.hgemm_adamw_load, "m ms v vs mo vo n".split(),
                  dict(m=A[0], ms=A[1], v=A[2], vs=A[3], mo=A[4], vo=A[5], n=100))
    for kw in (dict(n=-1), dict(ms=None), dict(mo=None), dict(m=None), dict(v=None), dict(vs=None), dict(vo=None),
               dict(ms=A[1] + 2), dict(mo=A[4] + 1), dict(m=None, ms=None, mo=None, v=None, vs=None, vo=None)):
        assert call(**kw) == BAD, kw
    for kw in (dict(mo=A[0]), dict(vo=A[1]), dict(vo=A[4] + 4), dict(mo=A[3])):
        assert call(**kw) == ALIAS, kw
    assert call(n=0) == OK


def test_experts(lib):
    size = tc.hgemm_experts_workspace_size
    need = size(16, 64, 32, 8, 2)
    assert need > 0
    for bad in ((-1, 64, 32, 8, 2), (65, 64, 32, 8, 2), (16, -1, 32, 8, 2), (16, 64, (1 << 20) + 1, 8, 2),
                (16, 64, 32, 0, 1), (16, 64, 32, 513, 2), (16, 64, 32, 8, 9), (16, 64, 32, 8, 0), (16, 64, 32, 64, 17)):
        assert size(*bad) == 0, bad
    names = ("X ldx Wr ldwr W1 ldw1 b1 W2 ldw2 b2 act gated k normalize R ldr Y ldy chosen share ws bytes M D F "
             "E").split()
    call = caller(lib.hgemm_experts, names,
                  dict(X=A[0], ldx=64, Wr=A[1], ldwr=64, W1=A[2], ldw1=64, b1=A[3], W2=A[4], ldw2=32, b2=A[5], act=3,
                       gated=1, k=2, normalize=1, R=A[6], ldr=64, Y=A[7], ldy=64, chosen=A[8], share=A[9], ws=A[10],
                       bytes=need, M=16, D=64, F=32, E=8))
    for kw in (dict(M=-1), dict(M=65), dict(k=0), dict(k=9), dict(E=0), dict(act=5), dict(act=-1), dict(gated=2),
               dict(normalize=-1), dict(X=None), dict(Wr=None), dict(W1=None), dict(W2=None), dict(Y=None),
               dict(ldx=63), dict(ldwr=63), dict(ldw1=63), dict(ldw2=31), dict(ldr=63), dict(ldy=63),
               dict(X=A[0] + 1), dict(chosen=A[8] + 2), dict(share=A[9] + 1), dict(ws=None), dict(ws=A[10] + 4),
               dict(bytes=need - 1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(Y=A[0]), dict(Y=A[2]), dict(Y=A[6] + 2), dict(Y=A[6], ldy=72), dict(chosen=A[7]), dict(share=A[8]),
               dict(share=A[6]), dict(ws=A[0]), dict(ws=A[4]), dict(ws=A[9]), dict(ws=A[7]), dict(Y=A[5]),
               dict(W2=A[2], Y=A[2])):
        assert call(**kw) == ALIAS, kw
    assert call(M=0) == OK


def test_binding_types():
    torch = pytest.importorskip("torch")
    h, f = torch.zeros(4, 4, dtype=torch.float16), torch.zeros(4, 4)
    with pytest.raises(TypeError):
        tc.hgemm_residual_norm_forward(f, 4, 1.0, h, 4, None, 2, h, None, 0, None, None, 1e-5, h, 4, None, 0, None, 4,
                                       4, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        tc.hgemm_experts(h, 4, h, 4, h, 4, None, h, 4, None, 0, False, 1, True, None, 0, h, 4, None, None, A[0], 4, 4,
                         4, 1, workspace_bytes=1 << 20, stream=0)
    for name, workspace in (("tensor", torch.zeros(1 << 20, dtype=torch.uint8)),):
        with pytest.raises(ValueError, match="workspace"):
            tc.hgemm_experts(A[0], 4, A[1], 4, A[2], 4, None, A[3], 4, None, 0, False, 1, True, None, 0, A[4], 4, None,
                             None, workspace, 4, 4, 4, 1, stream=0)
        with pytest.raises(ValueError, match="workspace"):
            tc.hgemm_residual_norm_backward(A[0], 4, A[1], 4, A[2], 4, A[3], 4, 1.0, None, 2, A[4], None, 2, A[5], A[6],
                                            A[7], 4, A[8], 4, None, None, None, None, None, workspace, 4, 4, stream=0)
    with pytest.raises(ValueError, match="grad is missing"):
        tc.hgemm_adamw_tensors([dict(weight=h, m=f, v=f)])
    with pytest.raises(TypeError, match="unknown"):
        tc.hgemm_adamw_tensors([dict(weight=h, grad=h, m=f, v=f, momentum=f)])
    with pytest.raises(ValueError, match="CUDA"):
        tc.hgemm_adamw_tensors([dict(weight=h, grad=h, m=f, v=f)])
    with pytest.raises(tc.HgemmError) as err:
        tc.hgemm_adamw_check(tc.AdamwTensors(table(adamw_tensor(m=A[0])), []))
    assert err.value.status == ALIAS
    with pytest.raises(TypeError):
        tc.hgemm_adamw_tensors([dict(weight=f, grad=h, m=f, v=f)])
    with pytest.raises(ValueError, match="dynamic"):
        tc.hgemm_adamw(tc.AdamwTensors(table(), []), 1e-3, dynamic=torch.zeros(16, dtype=torch.uint8), stream=0)


def test_dynamic_bytes():
    torch = pytest.importorskip("torch")
    b = tc.hgemm_adamw_dynamic(0.5, 2.0, 7, True)
    assert b.dtype == torch.uint8 and b.view(torch.float32)[:2].tolist() == [0.5, 2.0]
    assert b.view(torch.int32)[2:].tolist() == [7, 1]


def test_constants_match_the_header(lib):
    text = open(os.path.join(tcbuild.INCLUDE, "hgemm.h"), encoding="utf-8").read()
    found = re.findall(r"#define\s+(HGEMM_(?:NORM|TYPE|EXPERTS)_\w+|HGEMM_EXPERTS_MAX)\s+\(?([\d <]+)\)?", text)
    assert len(found) == 9, found
    for name, val in found:
        assert getattr(tc, name) == eval(val)  # noqa: S307 (a number, or one shifted)
    assert isinstance(lib, ctypes.CDLL) and ctypes.sizeof(tc._AdamwTensor) == 72
