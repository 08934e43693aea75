"""Host validation of the router, the combine's gradient, the dense product and the transposing quantiser (CPU only):
a refused call returns its status before anything is launched; the binding refuses wrong tensors."""

import ctypes

import pytest
import torch

import int4_weights_amd as moe

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, HIP, WORKSPACE = range(7)
P = 1 << 20  # a fake, aligned address: never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def _p(v):
    return ctypes.c_void_p(v)


def _topk(lib, **kw):
    a = dict(logits=P, type=0, ld=256, bias=None, T=4, E=256, k=8, score=1, G=8, TG=4, gtop=2, norm=1, scale=2.5, ids=P,
             w=P)
    a.update(kw)
    return lib.moe_router_topk(_p(a["logits"]), a["type"], a["ld"], _p(a["bias"]), a["T"], a["E"], a["k"], a["score"],
                               a["G"], a["TG"], a["gtop"], a["norm"], a["scale"], _p(a["ids"]), _p(a["w"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE),
    (dict(E=4, G=1, TG=1, k=5), SHAPE), (dict(type=2), UNSUPPORTED), (dict(score=2), UNSUPPORTED),
    (dict(scale=float("nan")), UNSUPPORTED), (dict(scale=float("inf")), UNSUPPORTED), (dict(ld=255), SHAPE),
    (dict(G=0), SHAPE), (dict(G=65), SHAPE), (dict(G=7), SHAPE), (dict(TG=0), SHAPE), (dict(TG=9), SHAPE),
    (dict(gtop=3), UNSUPPORTED), (dict(gtop=0), UNSUPPORTED), (dict(TG=1, k=33), SHAPE), (dict(logits=None), NULL),
    (dict(ids=None), NULL), (dict(w=None), NULL), (dict(logits=P + 2), ALIGN), (dict(bias=P + 2), ALIGN),
    (dict(ids=P + 1), ALIGN), (dict(T=0, logits=None, ids=None, w=None), OK), (dict(T=1 << 30), SHAPE),
])
def test_router_refusals(lib, kw, status):
    assert _topk(lib, **kw) == status
    assert (lib.moe_last_error() == b"") == (status == OK)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(type=5), UNSUPPORTED), (dict(score=-1), UNSUPPORTED),
    (dict(ld=10), SHAPE), (dict(ldd=10), SHAPE), (dict(d=None), NULL), (dict(dw=None), NULL), (dict(d=P + 1), ALIGN),
    (dict(T=0, d=None), OK),
])
def test_router_gradient_refusals(lib, kw, status):
    a = dict(type=0, ld=16, T=2, k=2, score=0, dw=P, d=P, ldd=16)
    a.update(kw)
    assert lib.moe_router_topk_bwd(_p(P), a["type"], a["ld"], _p(P), _p(a["dw"]), a["T"], 16, a["k"], a["score"], 1,
                                   1.0, _p(a["d"]), a["ldd"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(k=65), SHAPE), (dict(N=0), SHAPE), (dict(N=12), UNSUPPORTED), (dict(y_rows=-1), SHAPE),
    (dict(dY=None, dw=None), NULL), (dict(dZ=None), NULL), (dict(oi=None), NULL), (dict(w=None), NULL),
    (dict(Y=None), NULL), (dict(dZ=P + 8), ALIGN), (dict(dY=P + 8), ALIGN), (dict(T=1024, ws=None), WORKSPACE),
    (dict(T=1024, wsb=8 * 10000 - 1), WORKSPACE), (dict(T=1024, ws=P + 4), WORKSPACE), (dict(T=0), OK),
    (dict(T=0, y_rows=0, dZ=None, Y=None, oi=None, w=None, dY=None, dw=None, ws=None), OK),  # all empty
])
def test_combine_gradient_refusals(lib, kw, status):
    a = dict(dZ=P, Y=P, y_rows=10000, oi=P, w=P, T=512, k=8, N=64, dY=P, dw=P, ws=P, wsb=8 * 10000)
    a.update(kw)
    assert lib.moe_unpermute_combine_bwd(_p(a["dZ"]), _p(a["Y"]), a["y_rows"], _p(a["oi"]), _p(a["w"]), a["T"], a["k"],
                                         a["N"], _p(a["dY"]), _p(a["dw"]), _p(a["ws"]), a["wsb"], None) == status


def test_combine_gradient_workspace():
    assert moe.moe_unpermute_combine_bwd_workspace_bytes(512, 8, 10000) == 0
    assert moe.moe_unpermute_combine_bwd_workspace_bytes(513, 8, 10000) == 80000
    assert moe.moe_unpermute_combine_bwd_workspace_bytes(-1, 8, 10000) == -1
    assert moe.moe_unpermute_combine_bwd_workspace_bytes(1, 65, 10) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(M=1 << 30), SHAPE), (dict(K=100), UNSUPPORTED),
    (dict(gran=64), UNSUPPORTED), (dict(out=3), UNSUPPORTED), (dict(C=P, out=1), UNSUPPORTED), (dict(lda=240), SHAPE),
    (dict(ldw=128), SHAPE), (dict(ldd=99), SHAPE), (dict(C=P, ldc=99), SHAPE), (dict(lda=1 << 23), UNSUPPORTED),
    (dict(M=1 << 29, N=1 << 29, ldd=1 << 29), UNSUPPORTED), (dict(A=None), NULL), (dict(SFW=None), NULL),
    (dict(D=None), NULL), (dict(A=P + 8), ALIGN), (dict(lda=264), ALIGN), (dict(D=P + 2), ALIGN),
    (dict(SFA=P + 2), ALIGN), (dict(C=P, ldc=100, ldd=104), SHAPE), (dict(M=0, A=None, D=None), OK),
])
def test_dense_product_refusals(lib, kw, status):
    a = dict(A=P, lda=256, SFA=P, W=P, ldw=256, SFW=P, gran=128, D=P, out=0, ldd=100, C=None, ldc=100, M=300, N=100,
             K=256)
    a.update(kw)
    assert lib.moe_gemm_fp8(_p(a["A"]), a["lda"], _p(a["SFA"]), _p(a["W"]), a["ldw"], _p(a["SFW"]), a["gran"],
                            _p(a["D"]), a["out"], a["ldd"], _p(a["C"]), a["ldc"], a["M"], a["N"], a["K"], None, 0,
                            None) == status


@pytest.mark.parametrize("M,N", [((1 << 28) + 1, 1), (1, (1 << 28) + 1), (1 << 28, 256), (1 << 17, 1 << 19)])
def test_dense_product_too_large_for_one_launch(lib, M, N):
    assert lib.moe_gemm_fp8(_p(P), 128, _p(P), _p(P), 128, _p(P), 128, _p(P), 1, N, None, 0, M, N, 128, None, 0,
                            None) == UNSUPPORTED
    assert moe.moe_gemm_fp8_workspace_bytes(M, N, 128) == -1


@pytest.mark.parametrize("M,K", [(1 << 31, 8), (1 << 20, 1 << 17)])
def test_transposing_quantiser_too_large_for_one_launch(lib, M, K):
    assert lib.moe_quant_act_t(_p(P), M, K, K, _p(P), _p(P), None) == UNSUPPORTED


def test_dense_product_workspace(lib):
    assert moe.moe_gemm_fp8_workspace_bytes(4, 4, 100) == -1
    assert moe.moe_gemm_fp8_workspace_bytes(-1, 4, 128) == -1
    assert moe.moe_gemm_fp8_workspace_bytes(8192, 8192, 128) == 0
    # where a workspace is needed, a missing, short or misaligned one is refused
    for m, n, k in ((1, 64, 7168), (16, 256, 7168), (131, 7168, 2048), (64, 512, 32768)):
        need = moe.moe_gemm_fp8_workspace_bytes(m, n, k)
        assert need >= 0
        if need:
            for ws, size in ((None, need), (P, need - 1), (P + 4, need)):
                assert lib.moe_gemm_fp8(_p(P), k, _p(P), _p(P), k, _p(P), 128, _p(P), 0, n, None, 0, m, n, k, _p(ws), size,
                                        None) == WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=12, ld=16), UNSUPPORTED), (dict(ld=56), SHAPE),
    (dict(ld=68), ALIGN), (dict(x=None), NULL), (dict(q=P + 8), ALIGN), (dict(x=P + 8), ALIGN), (dict(s=P + 2), ALIGN),
    (dict(M=1 << 39), UNSUPPORTED), (dict(M=0, x=None, q=None, s=None), OK),
])
def test_transposing_quantiser_refusals(lib, kw, status):
    a = dict(x=P, M=5, K=64, ld=64, q=P, s=P)
    a.update(kw)
    assert lib.moe_quant_act_t(_p(a["x"]), a["M"], a["K"], a["ld"], _p(a["q"]), _p(a["s"]), None) == status


def test_binding_refuses_host_tensors():
    f = torch.zeros(2, 16)
    i = torch.zeros(2, 2, dtype=torch.int32)
    b = torch.zeros(2, 128, dtype=torch.bfloat16)
    u = torch.zeros(2, 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_router_topk(f, i, f[:, :2].contiguous())
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_router_topk_bwd(f, i, f, f)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_unpermute_combine_bwd(b, b, i, f, b, f)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_gemm_fp8(u, f, u, f, b)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_quant_act_t(b, u, f)
