"""moe_gemm_bf16's epilogues on every tile, whole, with edges and joined from shares of K (test_linear_epilogue_plan.py), plain and gated;
products in the gradients' orders in shares."""

import pytest
import torch

import int4_weights_amd as moe
from gpu_helpers import DEV, require_gpu
from linear_epilogue_shapes import EPILOGUES, SHARES
from test_gpu_gemm_linear import ORDERS, bf, check, make, strided

pytestmark = pytest.mark.gpu


def guarded(M, N, K):
    """(workspace or None, the bytes behind it)."""
    n = moe.moe_gemm_bf16_workspace_bytes(M, N, K)
    room = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    return (room[:n] if n else None), room[n:]


def sample(M):
    """Rows that the oracle computes: all of few, of many every 7th (each place of a tile's rows) and the last ones."""
    return list(range(M)) if M <= 300 else sorted({*range(0, M, 7), *range(M - 20, M)})


@pytest.mark.parametrize("shape", EPILOGUES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("gated,act", [(False, "gelu"), (False, "none"), (True, "silu"), (True, "gelu_tanh")])
@pytest.mark.parametrize("types", [("bf16", "fp32", "bf16"), ("fp32", "bf16", "fp32")])
def test_epilogues(shape, gated, act, types):
    require_gpu()
    M, N, K = shape
    out, btype, ctype = ({"bf16": torch.bfloat16, "fp32": torch.float32}[t] for t in types)
    A, W, a, w = make("nt", M, N, K, M + K, scale=K ** -0.5)
    g = torch.Generator().manual_seed(2)
    h = N // 2 if gated else N
    bias, C = torch.randn(N, generator=g).to(btype).to(DEV), torch.randn(M, h, generator=g).to(ctype).to(DEV)
    (rd, D), (rp, pre) = strided(torch.empty(M, h, dtype=out, device=DEV), 3, 5.0), strided(torch.empty(M, N, dtype=torch.bfloat16, device=DEV), 7, 9.0)
    ws, behind = guarded(M, N, K)
    moe.moe_gemm_bf16(A, W, D, bias=bias, act=act, gated=gated, C=C, pre=pre, workspace=ws)
    r = sample(M)
    check(D[r], a[r], w, bias, act, gated, C[r], pre[r])
    assert torch.isfinite(D).all() and torch.isfinite(pre).all()
    assert (rd[:, h:] == 5).all() and (rp[:, N:] == 9).all() and (behind == 0xA5).all()
    E = C.clone() if ctype is out else torch.empty_like(C, dtype=out)  # over the addend where it has D's type, pre not kept
    moe.moe_gemm_bf16(A, W, E, bias=bias, act=act, gated=gated, C=E if ctype is out else C, workspace=ws)
    assert torch.equal(E, D)


@pytest.mark.parametrize("order,shape", [(o, s) for o in SHARES for s in SHARES[o]], ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_in_shares(order, shape, out):
    require_gpu()
    M, N, K = shape
    A, W, a, w = make(order, M, N, K, M)
    ta, tw = ORDERS[order]
    C = bf(torch.Generator().manual_seed(4), M, N).to(out)
    D = C.clone()
    ws, behind = guarded(M, N, K)
    moe.moe_gemm_bf16(A, W, D, C=D, trans_a=ta, trans_w=tw, workspace=ws)
    r = sample(M)
    check(D[r], a[r], w, None, "none", False, C[r])
    assert (behind == 0xA5).all()
