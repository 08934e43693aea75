"""Host validation of moe_experts_decode (CPU only): a refused call returns its status before anything is launched."""

import ctypes

import pytest
import torch

import int4_weights_amd as moe

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, HIP, WORKSPACE = range(7)
P = 1 << 20  # a fake, aligned address: never dereferenced on these paths


def _p(v):
    return ctypes.c_void_p(v)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=4), UNSUPPORTED), (dict(fmt=3, s13=None), NULL), (dict(fmt=-1), UNSUPPORTED), (dict(fmt=0x20), UNSUPPORTED), (dict(T=-1), SHAPE),
    (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(H=0), SHAPE), (dict(I=0), SHAPE),
    (dict(T=129, k=1), UNSUPPORTED), (dict(T=128, k=9), UNSUPPORTED), (dict(T=1 << 30, k=64), UNSUPPORTED),
    (dict(H=192), UNSUPPORTED), (dict(I=64), UNSUPPORTED), (dict(H=32768 + 128), UNSUPPORTED), (dict(I=32768 + 128), UNSUPPORTED),
    (dict(x=None), NULL), (dict(ids=None), NULL), (dict(p=None), NULL), (dict(w13=None), NULL), (dict(w2=None), NULL),
    (dict(z=None), NULL), (dict(s13=None), NULL), (dict(s2=None), NULL), (dict(fmt=0), UNSUPPORTED),
    (dict(fmt=0, s13=None), UNSUPPORTED), (dict(x=P + 8), ALIGN), (dict(w13=P + 8), ALIGN), (dict(w2=P + 8), ALIGN),
    (dict(s13=P + 2), ALIGN), (dict(fmt=2, s2=P + 2), ALIGN), (dict(ids=P + 2), ALIGN), (dict(p=P + 2), ALIGN),
    (dict(z=P + 1), ALIGN), (dict(c=P + 1), ALIGN), (dict(status=P + 2), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(wsb=4 * 8 * 256 * 2 - 1), WORKSPACE), (dict(ws=P + 8), WORKSPACE),
    (dict(T=0, x=None, ids=None, p=None, w13=None, w2=None, z=None, s13=None, s2=None, ws=None), OK),
])
def test_refusals(kw, status):
    a = dict(fmt=1, x=P, ids=P, p=P, T=4, k=8, E=16, H=512, I=256, w13=P, s13=P, w2=P, s2=P, c=None, z=P, status=None, ws=P,
             wsb=4 * 8 * 256 * 2)
    a.update(kw)
    lib = moe.load()
    assert lib.moe_experts_decode(a["fmt"], _p(a["x"]), _p(a["ids"]), _p(a["p"]), a["T"], a["k"], a["E"], a["H"], a["I"],
                                  _p(a["w13"]), _p(a["s13"]), _p(a["w2"]), _p(a["s2"]), _p(a["c"]), _p(a["z"]),
                                  _p(a["status"]), _p(a["ws"]), a["wsb"], None) == status
    assert (lib.moe_last_error() == b"") == (status == OK)


def test_workspace_size():
    f = moe.moe_experts_decode_workspace_bytes
    assert f(4, 8, 256) == 4 * 8 * 256 * 2 and f(0, 8, 256) == 0
    assert f(-1, 8, 256) == f(129, 1, 256) == f(128, 9, 256) == f(1, 65, 256) == f(1, 1, 0) == f(1, 1, 32769) == -1


def test_binding_refuses_cpu_tensors_and_unknown_formats():
    t = torch.zeros(2, 128, dtype=torch.bfloat16)
    ids, p = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    w13, w2 = torch.zeros(1, 256, 128, dtype=torch.bfloat16), torch.zeros(1, 128, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_experts_decode(t, ids, p, w13, w2, t, weights="bf16")
    with pytest.raises(ValueError, match="one of bf16, fp8, int4, fp4"):
        moe.moe_experts_decode(t, ids, p, w13, w2, t, weights="int8")
