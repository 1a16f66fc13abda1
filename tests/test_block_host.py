"""Argument checks of the feed-forward block's operators (CPU: no computing
call is made; addresses are made up)."""

import ctypes

import pytest

import tensor_core_dense_fp16_gb300 as tc
from tensor_core_dense_fp16_gb300 import build as tcbuild

BAD, ALIAS, OK = tc.HGEMM_ERR_INVALID_ARG, tc.HGEMM_ERR_ALIAS, tc.HGEMM_OK
A = [0x10000000 * (i + 1) for i in range(10)]  # 16-byte aligned, disjoint


@pytest.fixture(scope="module")
def lib():
    tcbuild.build()
    return tc.load()


def caller(fn, names, defaults):
    def call(**kw):
        args = {**defaults, **kw}
        assert set(args) == set(names), set(args) ^ set(names)
        return fn(*[args[n] for n in names], None)
    return call


def linear(lib):
    names = "X ldx W ldw bias act R ldr Y ldy codes ldq scales lds M N K".split()
    return caller(lib.hgemm_linear, names,
                  dict(X=A[0], ldx=64, W=A[1], ldw=64, bias=A[2], act=2, R=A[3], ldr=128, Y=A[4], ldy=128,
                       codes=A[5], ldq=128, scales=A[6], lds=16, M=16, N=128, K=64))


def test_linear(lib):
    call = linear(lib)
    for kw in (dict(M=-1), dict(N=1 << 31), dict(K=1 << 40), dict(act=5), dict(act=-1), dict(ldx=63), dict(ldw=63),
               dict(ldr=127), dict(ldy=127), dict(ldq=127), dict(lds=15), dict(X=None), dict(W=None), dict(Y=None),
               dict(codes=None), dict(scales=None), dict(X=A[0] + 1), dict(bias=A[2] + 1), dict(scales=A[6] + 2),
               dict(ldx=1 << 41)):
        assert call(**kw) == BAD, kw
    y_bytes = 2 * 16 * 128
    for kw in (dict(Y=A[0]), dict(Y=A[1] + 2 * 8), dict(Y=A[2] - y_bytes + 2), dict(Y=A[3] + 2), dict(Y=A[3], ldy=136),
               dict(codes=A[4]), dict(codes=A[0]), dict(scales=A[5]), dict(scales=A[4]), dict(codes=A[3]),
               dict(X=A[4], R=A[4])):
        assert call(**kw) == ALIAS, kw
    # nothing to do; pointers of empty matrices may be null
    assert call(M=0) == OK and call(M=0, X=None, Y=None, R=None, codes=None, scales=None) == OK
    assert call(N=0) == OK


def test_dgrad(lib):
    names = "dY lddy W ldw codes ldq scales lds act dU lddu H ldh M N K".split()
    call = caller(lib.hgemm_linear_dgrad, names,
                  dict(dY=A[0], lddy=64, W=A[1], ldw=128, codes=A[2], ldq=128, scales=A[3], lds=16, act=2, dU=A[4],
                       lddu=128, H=A[5], ldh=128, M=16, N=64, K=128))
    for kw in (dict(M=-1), dict(lddy=63), dict(ldw=127), dict(ldq=127), dict(lds=15), dict(lddu=127), dict(ldh=127),
               dict(act=7), dict(codes=None), dict(codes=None, scales=None), dict(codes=None, scales=None, act=0),
               dict(dY=None), dict(dU=None), dict(H=A[5] + 1), dict(scales=A[3] + 1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dU=A[0]), dict(dU=A[2]), dict(H=A[4]), dict(H=A[1]), dict(H=A[3])):
        assert call(**kw) == ALIAS, kw
    assert call(M=0) == OK and call(K=0) == OK


def test_wgrad(lib):
    names = "dY lddy X ldx dW lddw dbias accumulate M N K".split()
    call = caller(lib.hgemm_linear_wgrad, names,
                  dict(dY=A[0], lddy=64, X=A[1], ldx=128, dW=A[2], lddw=128, dbias=A[3], accumulate=0, M=16, N=64,
                       K=128))
    for kw in (dict(N=-1), dict(lddy=63), dict(ldx=127), dict(lddw=127), dict(dY=None), dict(X=None), dict(dW=None),
               dict(dbias=A[3] + 2), dict(dW=A[2] + 1)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dW=A[0]), dict(dW=A[1]), dict(dbias=A[2]), dict(dbias=A[0])):
        assert call(**kw) == ALIAS, kw
    assert call(N=0) == OK


def test_layernorm(lib):
    names = "X ldx gamma beta eps Y ldy mean rstd M D".split()
    call = caller(lib.hgemm_layernorm_forward, names,
                  dict(X=A[0], ldx=64, gamma=A[1], beta=A[2], eps=1e-5, Y=A[3], ldy=64, mean=A[4], rstd=A[5], M=16,
                       D=64))
    for kw in (dict(M=-1), dict(ldx=63), dict(ldy=63), dict(gamma=None), dict(beta=None), dict(X=None), dict(Y=None),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(mean=None), dict(rstd=None),
               dict(mean=A[4] + 2)):
        assert call(**kw) == BAD, kw
    for kw in (dict(Y=A[0] + 2), dict(Y=A[0], ldy=72), dict(Y=A[1]), dict(mean=A[5]), dict(mean=A[0]),
               dict(rstd=A[3])):
        assert call(**kw) == ALIAS, kw
    assert call(M=0) == OK and call(D=0) == OK

    size = tc.hgemm_layernorm_backward_workspace_size
    need = size(16, 64)
    assert need > 0 and size(0, 0) == 0 and size(-1, 64) == 0
    assert size(16384, 8192) <= 1024 * 2 * (8192 + 32) * 4
    names = "dY lddy X ldx gamma mean rstd R ldr dX lddx dgamma dbeta ws bytes M D".split()
    call = caller(lib.hgemm_layernorm_backward, names,
                  dict(dY=A[0], lddy=64, X=A[1], ldx=64, gamma=A[2], mean=A[3], rstd=A[4], R=A[5], ldr=64, dX=A[6],
                       lddx=64, dgamma=A[7], dbeta=A[8], ws=A[9], bytes=need, M=16, D=64))
    for kw in (dict(M=-1), dict(lddy=63), dict(ldx=63), dict(ldr=63), dict(lddx=63), dict(gamma=None), dict(mean=None),
               dict(rstd=None), dict(dgamma=None), dict(dbeta=None), dict(ws=None), dict(bytes=need - 1),
               dict(ws=A[9] + 8), dict(dX=None)):
        assert call(**kw) == BAD, kw
    for kw in (dict(dX=A[1]), dict(dX=A[0] + 2), dict(dX=A[5], lddx=72), dict(dX=A[2]), dict(dgamma=A[8]),
               dict(ws=A[0]), dict(ws=A[7]), dict(dbeta=A[5]), dict(X=A[6], R=A[6])):
        assert call(**kw) == ALIAS, kw
    assert call(D=0) == OK


def test_ckpt8(lib):
    save = caller(lib.hgemm_ckpt8_save, "X ldx codes ldq scales lds M N".split(),
                  dict(X=A[0], ldx=128, codes=A[1], ldq=128, scales=A[2], lds=16, M=16, N=128))
    load = caller(lib.hgemm_ckpt8_load, "codes ldq scales lds act Y ldy M N".split(),
                  dict(codes=A[1], ldq=128, scales=A[2], lds=16, act=1, Y=A[0], ldy=128, M=16, N=128))
    for kw in (dict(M=-1), dict(ldq=127), dict(lds=15), dict(codes=None), dict(scales=None), dict(scales=A[2] + 1)):
        assert save(**kw) == BAD and load(**kw) == BAD, kw
    assert save(X=A[0] + 1) == BAD and load(act=9) == BAD and load(Y=None) == BAD
    for kw in (dict(codes=A[0]), dict(scales=A[0])):
        assert save(**kw) == ALIAS and load(**kw) == ALIAS, kw
    assert save(scales=A[1]) == ALIAS
    assert save(M=0) == OK and load(N=0) == OK


def test_binding_types():
    torch = pytest.importorskip("torch")
    h, f = torch.zeros(4, 4, dtype=torch.float16), torch.zeros(4, 4)
    with pytest.raises(TypeError):
        tc.hgemm_linear(f, 4, h, 4, None, 0, None, 0, h, 4, 4, 4, 4, stream=0)
    with pytest.raises(ValueError):
        tc.hgemm_linear(h, 4, h, 4, None, 0, None, 0, h, 4, 4, 4, 4, stream=0)
    with pytest.raises(TypeError):
        tc.hgemm_ckpt8_save(f, 4, h, 4, f, 4, 4, 4, stream=0)


def test_constants_match_the_header(lib):
    import os
    import re
    text = open(os.path.join(tcbuild.INCLUDE, "hgemm.h"), encoding="utf-8").read()
    found = re.findall(r"#define\s+(HGEMM_(?:ACT|CKPT8)_\w+)\s+(\d+)", text)
    assert len(found) == 6
    for name, val in found:
        assert getattr(tc, name) == int(val)
    assert isinstance(lib, ctypes.CDLL)
