"""Host validation of moe_gemm_bf16 and moe_act_bwd (CPU only): a refused call returns its status before anything is
launched; the binding refuses wrong tensors."""

import ctypes

import pytest
import torch

import int4_weights_amd as moe

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, HIP, WORKSPACE = range(7)
P = 1 << 20  # a fake, aligned address: never dereferenced on these paths
F32, BF16, GATED = 0, 1, 0x10
EMPTY = dict(A=None, W=None, D=None, M=0)


def _p(v):
    return ctypes.c_void_p(v)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=-8), SHAPE), (dict(M=(1 << 26) + 1), UNSUPPORTED),
    (dict(N=(1 << 26) + 1), UNSUPPORTED), (dict(M=1 << 20, N=1 << 20, ldd=1 << 20), UNSUPPORTED), (dict(tr=1), UNSUPPORTED), (dict(tr=4), UNSUPPORTED),
    (dict(act=5), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(act=0x20), UNSUPPORTED), (dict(act=GATED, N=255), UNSUPPORTED),
    (dict(act=GATED, tr=2), UNSUPPORTED), (dict(act=GATED, tr=3), UNSUPPORTED), (dict(out=2), UNSUPPORTED),
    (dict(bias=P, btype=2), UNSUPPORTED), (dict(C=P, ctype=-1), UNSUPPORTED), (dict(K=132), UNSUPPORTED),
    (dict(tr=2, K=132), UNSUPPORTED), (dict(tr=2, N=252), UNSUPPORTED), (dict(tr=3, M=68), UNSUPPORTED),
    (dict(tr=3, N=252), UNSUPPORTED), (dict(lda=127), SHAPE), (dict(ldw=127), SHAPE), (dict(tr=2, ldw=255), SHAPE),
    (dict(tr=3, lda=63, ldw=256), SHAPE), (dict(ldd=255), SHAPE), (dict(C=P, ldc=255), SHAPE), (dict(pre=P, ldp=255), SHAPE),
    (dict(act=GATED | 2, ldd=127), SHAPE), (dict(lda=1 << 22), UNSUPPORTED), (dict(ldw=1 << 22), UNSUPPORTED),
    (dict(act=GATED, N=1 << 12, ldd=1 << 12, ldw=(1 << 22) - 8), UNSUPPORTED),
    (dict(act=GATED, N=2, ldd=2, ldw=(1 << 22) - 8), UNSUPPORTED), (dict(EMPTY, act=GATED, N=510, ldd=255, ldw=1 << 21), OK), (dict(A=None), NULL), (dict(W=None), NULL),
    (dict(D=None), NULL), (dict(A=P + 8), ALIGN), (dict(W=P + 2), ALIGN), (dict(lda=132), ALIGN), (dict(ldw=130), ALIGN),
    (dict(D=P + 1), ALIGN), (dict(D=P + 2, out=F32), ALIGN), (dict(bias=P + 2, btype=F32), ALIGN), (dict(bias=P + 1, btype=BF16), ALIGN),
    (dict(C=P + 2, ctype=F32), ALIGN), (dict(pre=P + 1), ALIGN), (dict(C=P + 4096, D=P + 4096, ldc=264), SHAPE),
    (dict(C=P + 4096, D=P + 4096, ctype=F32), SHAPE), (dict(M=131, N=200, ldd=200, K=8192, lda=8192, ldw=8192, ws=None), WORKSPACE),
    (dict(M=131, N=200, ldd=200, K=8192, lda=8192, ldw=8192, wsb=1024), WORKSPACE),
    (dict(M=131, N=200, ldd=200, K=8192, lda=8192, ldw=8192, ws=P + 8), WORKSPACE), (EMPTY, OK), (dict(EMPTY, act=GATED | 2, ws=None), OK),
])
def test_product_refusals(kw, status):
    a = dict(A=P, lda=128, W=P, ldw=128, tr=0, D=P, out=BF16, ldd=256, bias=None, btype=F32, act=0, C=None, ctype=BF16, ldc=256,
             pre=None, ldp=256, M=64, N=256, K=128, ws=P, wsb=1 << 30)
    a.update(kw)
    lib = moe.load()
    got = lib.moe_gemm_bf16(_p(a["A"]), a["lda"], _p(a["W"]), a["ldw"], a["tr"], _p(a["D"]), a["out"], a["ldd"], _p(a["bias"]),
                            a["btype"], a["act"], _p(a["C"]), a["ctype"], a["ldc"], _p(a["pre"]), a["ldp"], a["M"], a["N"],
                            a["K"], _p(a["ws"]), a["wsb"], None)
    assert got == status
    assert (lib.moe_last_error() == b"") == (status == OK)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(M=(1 << 26) + 1), UNSUPPORTED), (dict(N=1 << 27), UNSUPPORTED), (dict(act=9), UNSUPPORTED),
    (dict(act=GATED, N=255), UNSUPPORTED), (dict(dP=None, db=None), NULL), (dict(dD=None), NULL),
    (dict(pre=None), NULL), (dict(pre=None, act=GATED), NULL), (dict(ldd=248), SHAPE), (dict(ldp=248), SHAPE), (dict(ldo=248), SHAPE),
    (dict(act=GATED | 2, ldd=120), SHAPE), (dict(dD=P + 1), ALIGN), (dict(pre=P + 1), ALIGN), (dict(dP=P + 1), ALIGN), (dict(db=P + 2), ALIGN),
    (dict(dD=P, dP=P, ldo=264), SHAPE),
    (dict(dD=P, dP=P, act=GATED | 2), SHAPE), (dict(dP=P + 65536, pre=P + 65536, ldp=264), SHAPE), (dict(M=2000, ws=None), WORKSPACE),
    (dict(M=2000, wsb=16), WORKSPACE), (dict(M=2000, ws=P + 4), WORKSPACE), (dict(M=0, dD=None, pre=None, dP=P, db=None), OK),
    (dict(M=0, dD=None, pre=None, dP=None, db=P, acc=1), OK),
])
def test_gradient_refusals(kw, status):
    a = dict(dD=P, ldd=256, pre=P + 4096, ldp=256, act=2, dP=P + 8192, ldo=256, db=P, acc=0, M=64, N=256, ws=P, wsb=1 << 30)
    a.update(kw)
    lib = moe.load()
    assert lib.moe_act_bwd(_p(a["dD"]), a["ldd"], _p(a["pre"]), a["ldp"], a["act"], _p(a["dP"]), a["ldo"], _p(a["db"]), a["acc"],
                           a["M"], a["N"], _p(a["ws"]), a["wsb"], None) == status
    assert (lib.moe_last_error() == b"") == (status == OK)


def test_workspace_sizes():
    f, g = moe.moe_gemm_bf16_workspace_bytes, moe.moe_act_bwd_workspace_bytes
    assert f(-1, 8, 8) == f(8, 0, 8) == f(8, 8, -1) == f(1 << 27, 8, 8) == f(1 << 20, 1 << 20, 8) == -1
    assert f(0, 8, 8) == 0 and f(8192, 8192, 4096) == 0 and f(131, 200, 8192) > 0
    assert g(-1, 8) == g(8, 0) == g(1 << 27, 8) == -1 and g(0, 8) == g(1024, 8) == 0 and g(1025, 8) == 33 * 8 * 4


def test_binding_refuses():
    x, w, d = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16), torch.zeros(4, 32)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_gemm_bf16(x, w, d)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_act_bwd(x, x, x)
    with pytest.raises(ValueError, match="one of none, relu"):
        from int4_weights_amd import _lib
        _lib._act("f", "tanh", False)
