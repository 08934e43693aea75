"""moe_act_bwd against the float64 oracle and against differences through moe_gemm_bf16."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def f64(t):
    return t.double().cpu().numpy()


def run(dD, pre, act, gated, dP=True, dbias=None, accumulate=False):
    M, h = dD.shape
    N = 2 * h if gated else h
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV) if dP is True else dP
    n = moe.moe_act_bwd_workspace_bytes(M, N)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n > 0 else None
    moe.moe_act_bwd(dD, pre, out, dbias=dbias, act=act, gated=gated, accumulate=accumulate, workspace=ws)
    return out


def inputs(M, N, gated, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    dD = torch.randn(M, N // 2 if gated else N, generator=g).to(torch.bfloat16).to(DEV)
    return dD, (torch.randn(M, N, generator=g) * scale).to(torch.bfloat16).to(DEV)


def check(dP, dbias, dD, pre, act, gated, before=0.0):
    ref = oracle.act_bwd(f64(dD), f64(pre), act, gated)
    # the functions to 2^-18 of their terms (exponents of up to 32, see the product's test), which near a slope's zero are
    # larger than it: silu' and gelu' are sums of terms up to |v| / 2; then half a step of bf16
    mag = np.abs(f64(dD)) * (1 + np.abs(f64(pre)[:, :dD.shape[1]]))
    if gated:
        mag = np.concatenate((mag * np.abs(f64(pre)[:, dD.shape[1]:]), mag), 1)
    err = (0 if act == "none" and not gated else 2.0 ** -18) * mag
    if dP is not None:
        assert (np.abs(f64(dP) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err) + 1e-37).all()
    if dbias is not None:
        bound = err.sum(0) + 2 * (dD.shape[0] + 2) * 2.0 ** -24 * (np.abs(ref).sum(0) + np.abs(before))
        assert (np.abs(f64(dbias) - before - ref.sum(0)) <= bound + 1e-37).all()


@pytest.mark.parametrize("shape", [(1, 2), (1, 16), (5, 34), (3, 80), (17, 528), (700, 2344), (333, 1536), (1000, 1042), (1500, 1170), (2050, 4096)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_against_the_oracle(shape, act, gated):
    require_gpu()
    M, N = shape
    dD, pre = inputs(M, N, gated, M + N)
    db = torch.full((N,), 7.0, device=DEV)
    dP = run(dD, pre, act, gated, dbias=db)
    check(dP, db, dD, pre, act, gated)
    again, db2 = torch.empty_like(dP), torch.empty_like(db)
    run(dD, pre, act, gated, dP=again, dbias=db2)
    assert torch.equal(dP, again) and torch.equal(db, db2)
    assert torch.equal(run(dD, pre, act, gated), dP)  # without a bias
    db3 = torch.empty_like(db)
    run(dD, pre, act, gated, dP=None, dbias=db3)
    assert torch.equal(db3, db)


def test_bias_alone_and_accumulated():
    require_gpu()
    dD, _ = inputs(700, 264, False, 1)
    before = torch.randn(264, generator=torch.Generator().manual_seed(1)).to(DEV)
    db = before.clone()
    run(dD, None, "none", False, dP=None, dbias=db, accumulate=True)
    check(None, db, dD, dD, "none", False, f64(before))
    db = before[:16].clone()
    few, _ = inputs(5, 16, False, 2)
    run(few, None, "none", False, dP=None, dbias=db, accumulate=True)
    check(None, db, few, few, "none", False, f64(before)[:16])


def test_no_rows():
    require_gpu()
    e = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    db = torch.full((16,), 3.0, device=DEV)
    run(e, e, "silu", False, dbias=db, accumulate=True)
    assert (db == 3).all()
    run(e, e, "silu", False, dbias=db)
    assert (db == 0).all()


@pytest.mark.parametrize("gated", [False, True])
def test_strided_and_in_place(gated):
    require_gpu()
    M, N = 130, 272
    dD, pre = inputs(M, N, gated, 4)
    want = run(dD, pre, "gelu", gated)
    h = dD.shape[1]
    a, b, c = (torch.full((M, w + 3 * i), 5.0, dtype=torch.bfloat16, device=DEV) for i, w in ((1, h), (2, N), (3, N)))
    a[:, :h], b[:, :N] = dD, pre
    moe.moe_act_bwd(a[:, :h], b[:, :N], c[:, :N], act="gelu", gated=gated)
    assert torch.equal(c[:, :N], want) and (c[:, N:] == 5).all()
    p = pre.clone()
    run(dD, p, "gelu", gated, dP=p)  # over the pre-activation
    assert torch.equal(p, want)
    if not gated:
        d = dD.clone()
        run(d, pre, "gelu", gated, dP=d)
        assert torch.equal(d, want)


def test_a_bad_value_stays_in_its_column():
    require_gpu()
    dD, pre = inputs(300, 64, False, 5)
    db = torch.empty(64, device=DEV)
    dP = run(dD, pre, "silu", False, dbias=db)
    dD[200, 9] = float("nan")
    db2 = torch.empty(64, device=DEV)
    dP2 = run(dD, pre, "silu", False, dbias=db2)
    keep = torch.arange(64, device=DEV) != 9
    assert torch.equal(db[keep], db2[keep]) and torch.isnan(db2[9]) and torch.equal(dP[:, keep], dP2[:, keep])
    assert torch.isnan(dP2[200, 9]) and torch.equal(dP[:200], dP2[:200])


def test_captured_and_replayed():
    require_gpu()
    M, N = 900, 528
    dD, pre = inputs(M, N, True, 6)
    dP, db = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(N, device=DEV)
    run(dD, pre, "silu", True, dP=dP, dbias=db)
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(moe.moe_act_bwd_workspace_bytes(M, N), dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(g):
        moe.moe_act_bwd(dD, pre, dP, dbias=db, act="silu", gated=True, workspace=ws)
    for i in range(4):
        d2, p2 = inputs(M, N, True, 10 + i)
        dD.copy_(d2), pre.copy_(p2)
        wb = torch.empty_like(db)
        want = run(d2, p2, "silu", True, dbias=wb)
        dP.zero_(), db.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dP, want) and torch.equal(db, wb)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients_against_differences(act, gated):
    """The chain (product, bias, activation; then act_bwd and the two products) against central differences of the float64
    chain, at the bf16 operands' values."""
    require_gpu()
    M, N, K = 9, 16, 24
    g = torch.Generator().manual_seed(7)
    x, w = (torch.randn(s, generator=g).to(torch.bfloat16).to(DEV) for s in ((M, K), (N, K)))
    b = torch.randn(N, generator=g).to(DEV)
    h = N // 2 if gated else N
    dy = torch.randn(M, h, generator=g).to(torch.bfloat16).to(DEV)
    y, pre = torch.empty(M, h, dtype=torch.bfloat16, device=DEV), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_bf16(x, w, y, bias=b, act=act, gated=gated, pre=pre)
    db, dx, dw = torch.empty(N, device=DEV), torch.empty(M, K, device=DEV), torch.empty(N, K, device=DEV)
    dP = run(dy, pre, act, gated, dbias=db)
    moe.moe_gemm_bf16(dP, w, dx, trans_w=True)
    # the contraction's length M = 9 is any; N and K are multiples of 8
    moe.moe_gemm_bf16(dP, x, dw, trans_a=True, trans_w=True)

    def loss(x, w, b):
        return (oracle.linear(x, w, b, act, gated)[0] * f64(dy)).sum()

    X, W, B = f64(x), f64(w), f64(b)
    # pre and dP are bf16: each half a step, 2^-8, of terms that are added up; slopes change by at most 1.2 |d pre| (times up)
    for got, at, n in ((dx, 0, 40), (dw, 1, 40), (db, 2, N)):
        args = [X, W, B]
        r = np.random.default_rng(at)
        num, val = [], []
        for _ in range(n):
            i = tuple(r.integers(0, s) for s in args[at].shape)
            p, m = [v.copy() for v in args], [v.copy() for v in args]
            p[at][i] += 1e-5
            m[at][i] -= 1e-5
            num.append((loss(*p) - loss(*m)) / 2e-5)
            val.append(f64(got)[i])
        num, val = np.array(num), np.array(val)
        # relative to the size of the whole gradient: the errors are independent of each entry's own size
        scale = np.abs(f64(got)).max()
        assert np.abs(num - val).max() < 4 * 2.0 ** -8 * scale, (at, np.abs(num - val).max() / scale)
