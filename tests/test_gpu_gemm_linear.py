"""moe_gemm_bf16 against the float64 oracle: every kernel, operand order, epilogue, type, odd sizes, strides; values outside
the matrices, rows behind them, workspaces, streams, graphs, offsets past 32 bits."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu
from linear_shapes import REACHED

pytestmark = pytest.mark.gpu

ORDERS = {"nt": (False, False), "nn": (False, True), "tn": (True, True)}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


def strided(t, pad, fill):
    """t as a view of wider rows whose rest holds `fill`."""
    room = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    room[:, :t.shape[1]] = t
    return room, room[:, :t.shape[1]]


def workspace(M, N, K):
    n = moe.moe_gemm_bf16_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=DEV) if n > 0 else None


def check(D, a, w, bias, act, gated, C, pre=None):
    """a [M, K], w [N, K] in float64.  Sums of K products (and the bias) in fp32, in any order: at most 2 (K + 2) * 2^-24 of
    their magnitudes.  The activations' slopes are at most 1.13; they are evaluated to 2^-18 of their value (an exponent of up
    to 32 rounded to fp32 is off by 32 * 2^-24, the functions by a few units in the last place).  Then one rounding."""
    ref, v, mag = oracle.linear(a, w, f64(bias), act, gated, f64(C))
    dv = 2.0 * (a.shape[1] + 2) * 2.0 ** -24 * mag
    e = 2.0 ** -18 if act != "none" else 0.0
    h = ref.shape[1]
    if gated:
        av = oracle.act(act, v[:, :h])
        err = (1.13 * dv[:, :h] + e * np.abs(av)) * (np.abs(v[:, h:]) + dv[:, h:]) + np.abs(av) * dv[:, h:] + 2.0 ** -23 * np.abs(av * v[:, h:])
    else:
        err = 1.13 * dv + e * np.abs(oracle.act(act, v))
    err += 0.0 if C is None else 2.0 ** -24 * (np.abs(f64(C)) + np.abs(ref))
    step = 2.0 ** -8 if D.dtype is torch.bfloat16 else 2.0 ** -24
    got = f64(D)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= err + step * (np.abs(ref) + err) + 1e-37).all(), float((np.abs(got - ref) - err).max())
    if pre is not None:
        assert (np.abs(f64(pre) - v) <= dv + 2.0 ** -8 * (np.abs(v) + dv) + 1e-37).all()


def make(order, M, N, K, seed=0, scale=0.3):
    g = torch.Generator().manual_seed(seed)
    ta, tw = ORDERS[order]
    A, W = bf(g, *((K, M) if ta else (M, K))), bf(g, *((K, N) if tw else (N, K)), scale=scale)
    return A, W, f64(A).T if ta else f64(A), f64(W).T if tw else f64(W)


CASES = [(o, s) for o in REACHED for s in REACHED[o]]  # every kernel (test_linear_plan.py)


@pytest.mark.parametrize("order,shape", CASES, ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products(order, shape, out):
    require_gpu()
    M, N, K = shape
    A, W, a, w = make(order, M, N, K, M + N + K)
    ta, tw = ORDERS[order]
    room, D = strided(torch.empty(M, N, dtype=out, device=DEV), 3, 5.0)
    moe.moe_gemm_bf16(A, W, D, trans_a=ta, trans_w=tw, workspace=workspace(M, N, K))
    check(D, a, w, None, "none", False, None)
    assert (room[:, N:] == 5).all()


@pytest.mark.parametrize("shape", [(1, 4096, 7168), (3, 2, 8), (16, 48, 200), (31, 262, 264), (64, 96, 520), (131, 264, 2048),
                                   (333, 1030, 512), (1100, 2304, 72), (2300, 4090, 104)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated(shape, act):
    require_gpu()
    M, N, K = shape
    A, W, a, w = make("nt", M, N, K, 3, scale=K ** -0.5)
    g = torch.Generator().manual_seed(1)
    bias, C = torch.randn(N, generator=g).to(DEV), bf(g, M, N // 2)
    _, D = strided(torch.empty(M, N // 2, dtype=torch.bfloat16, device=DEV), 5, 0.0)
    room, pre = strided(torch.empty(M, N, dtype=torch.bfloat16, device=DEV), 7, 9.0)
    moe.moe_gemm_bf16(A, W, D, bias=bias, act=act, gated=True, C=C, pre=pre, workspace=workspace(M, N, K))
    check(D, a, w, bias, act, True, C, pre)
    assert (room[:, N:] == 9).all()


@pytest.mark.parametrize("M", [2, 40, 70, 1200])  # streams, split and whole tiles
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("types", [("bf16", "fp32", "bf16"), ("fp32", "bf16", "fp32"), ("bf16", None, None)])
def test_epilogues(M, act, gated, types):
    require_gpu()
    out, btype, ctype = types
    N, K = 200, 1544
    t = {"bf16": torch.bfloat16, "fp32": torch.float32}
    A, W, a, w = make("nt", M, N, K, 5, scale=0.05)
    g = torch.Generator().manual_seed(2)
    h = N // 2 if gated else N
    bias = None if btype is None else torch.randn(N, generator=g).to(t[btype]).to(DEV)
    C = None if ctype is None else torch.randn(M, h, generator=g).to(t[ctype]).to(DEV)
    D = torch.empty(M, h, dtype=t[out], device=DEV)
    pre = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_bf16(A, W, D, bias=bias, act=act, gated=gated, C=C, pre=pre, workspace=workspace(M, N, K))
    check(D, a, w, bias, act, gated, C, pre)
    E = torch.empty_like(D)
    moe.moe_gemm_bf16(A, W, E, bias=bias, act=act, gated=gated, C=C, workspace=workspace(M, N, K))
    assert torch.equal(D, E)  # keeping pre changes nothing, and results repeat


@pytest.mark.parametrize("order,shape", [("nt", (9, 40, 136)), ("nt", (300, 264, 136)), ("nn", (300, 264, 136)),
                                         ("tn", (304, 264, 131)), ("nt", (2100, 2056, 72)), ("tn", (2104, 2056, 70))])
def test_what_lies_outside_is_not_read_as_values(order, shape):
    """Operands inside wider rows full of NaN; nothing of them reaches the product."""
    require_gpu()
    M, N, K = shape
    A, W, a, w = make(order, M, N, K, 8)
    (_, As), (_, Ws) = strided(A, 8, float("nan")), strided(W, 24, float("nan"))
    ta, tw = ORDERS[order]
    D = torch.empty(M, N, device=DEV)
    moe.moe_gemm_bf16(As, Ws, D, trans_a=ta, trans_w=tw, workspace=workspace(M, N, K))
    check(D, a, w, None, "none", False, None)


@pytest.mark.parametrize("order,M", [("nt", 12), ("nt", 200), ("nn", 200), ("tn", 200)])
def test_a_bad_value_stays_in_its_row_and_column(order, M):
    require_gpu()
    N, K = 136, 200
    A, W, _, _ = make(order, M, N, K, 4)
    ta, tw = ORDERS[order]
    D, E = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV)
    moe.moe_gemm_bf16(A, W, D, trans_a=ta, trans_w=tw, workspace=workspace(M, N, K))
    (A.t() if ta else A)[7, 100] = float("nan")
    (W.t() if tw else W)[33, 5] = float("inf")
    moe.moe_gemm_bf16(A, W, E, trans_a=ta, trans_w=tw, workspace=workspace(M, N, K))
    keep = torch.ones(M, N, dtype=torch.bool, device=DEV)
    keep[7], keep[:, 33] = False, False
    assert torch.equal(D[keep], E[keep]) and torch.isnan(E[7]).all() and not torch.isfinite(E[:, 33]).any()


@pytest.mark.parametrize("order,shape", [("tn", (264, 136, 500)), ("nt", (7, 40, 64)), ("nn", (1100, 1032, 64))])
def test_accumulates_in_place(order, shape):
    require_gpu()
    M, N, K = shape
    A, W, a, w = make(order, M, N, K, 6)
    ta, tw = ORDERS[order]
    D = torch.randn(M, N, generator=torch.Generator().manual_seed(3)).to(DEV)
    C = D.clone()
    moe.moe_gemm_bf16(A, W, D, C=D, trans_a=ta, trans_w=tw, workspace=workspace(M, N, K))
    check(D, a, w, None, "none", False, C)


def test_no_rows_and_no_products():
    require_gpu()
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    moe.moe_gemm_bf16(e(0, 64), e(40, 64), e(0, 40))
    C = torch.randn(24, 40, device=DEV)
    for M, order in ((24, "tn"), (24, "nt"), (24, "nn")):  # no tokens: the gradient stays
        ta, tw = ORDERS[order]
        D = C.clone()
        moe.moe_gemm_bf16(e(0, M) if ta else e(M, 0), e(0, 40) if tw else e(40, 0), D, C=D, trans_a=ta, trans_w=tw)
        assert torch.equal(D, C)
    bias = torch.randn(40, device=DEV)
    D = torch.empty(24, 40, device=DEV)
    moe.moe_gemm_bf16(e(24, 0), e(40, 0), D, bias=bias, act="relu")
    assert torch.equal(D, bias.clamp_min(0).expand(24, 40))


def test_limits_of_the_activations():
    """Far arguments: no NaN where the activation has a limit, and small results keep their relative precision."""
    require_gpu()
    v = torch.tensor([-3e38, -1e4, -60.0, -20.0, -9.0, -5.0, -1e-3, -0.0, 0.0, 1e-30, 1e-3, 9.0, 60.0, 1e4, 3e38])
    A = torch.zeros(1, 8, dtype=torch.bfloat16, device=DEV)
    W = torch.zeros(v.numel(), 8, dtype=torch.bfloat16, device=DEV)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        D = torch.empty(1, v.numel(), device=DEV)
        moe.moe_gemm_bf16(A, W, D, bias=v.to(DEV), act=act)
        x = v.double().numpy()
        with np.errstate(over="ignore"):
            ref = oracle.act(act, x)
        # exponents of up to 200 in fp32: 200 * 2^-23 relative; below the smallest normal number anything
        assert (np.abs(f64(D)[0] - ref) <= 200 * 2.0 ** -23 * np.abs(ref) + 2.0 ** -120).all(), act


def test_workspace_is_used_and_not_overrun():
    require_gpu()
    M, N, K = 131, 200, 8192
    n = moe.moe_gemm_bf16_workspace_bytes(M, N, K)
    assert n > 0
    A, W, a, w = make("nt", M, N, K, 2)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    D = torch.empty(M, N, device=DEV)
    moe.moe_gemm_bf16(A, W, D, workspace=ws[:n])
    check(D, a, w, None, "none", False, None)
    assert (ws[n:] == 0xA5).all()
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_gemm_bf16(A, W, D)


def test_streams_and_graph():
    require_gpu()
    M, N, K = 131, 200, 8192
    A, W, _, _ = make("nt", M, N, K, 2)
    B, V, _, _ = make("tn", 512, 264, 300, 3)
    D, E = torch.empty(M, N, device=DEV), torch.empty(512, 264, device=DEV)
    moe.moe_gemm_bf16(A, W, D, workspace=workspace(M, N, K))
    moe.moe_gemm_bf16(B, V, E, trans_a=True, trans_w=True, workspace=workspace(512, 264, 300))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = workspace(M, N, K), workspace(512, 264, 300)
    outs = [(torch.empty_like(D), torch.empty_like(E)) for _ in range(8)]
    torch.cuda.synchronize()
    for d, e in outs:
        moe.moe_gemm_bf16(A, W, d, workspace=w1, stream=s1)
        moe.moe_gemm_bf16(B, V, e, trans_a=True, trans_w=True, workspace=w2, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(d, D) and torch.equal(e, E) for d, e in outs)
    out = torch.empty_like(D)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_gemm_bf16(A, W, out, workspace=w1)
    for i in range(4):
        A2, _, a, w = make("nt", M, N, K, 10 + i)
        A.copy_(A2)
        want = torch.empty_like(D)
        moe.moe_gemm_bf16(A, W, want, workspace=workspace(M, N, K))
        out.fill_(1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("order", ["nt", "tn"])
def test_offsets_past_32_bits(order):
    """Operands and outputs that lie beyond 2^32 bytes of their first element."""
    require_gpu()
    ta, tw = ORDERS[order]
    if order == "nt":  # 2100 rows of A, 2 MB apart; of D, too
        M, N, K, ld = 2100, 136, 128, 1 << 20
        A = torch.empty(M, ld, dtype=torch.bfloat16, device=DEV)[:, :K]
        W = bf(torch.Generator().manual_seed(1), N, K)
    else:  # 2200 tokens, 2 MB apart
        M, N, K, ld = 64, 136, 2200, 1 << 20
        A = torch.empty(K, ld, dtype=torch.bfloat16, device=DEV)[:, :M]
        W = bf(torch.Generator().manual_seed(1), K, N)
    A.copy_(bf(torch.Generator().manual_seed(2), *A.shape))
    D = torch.empty(M, ld, device=DEV)[:, :N] if order == "nt" else torch.empty(M, N, device=DEV)
    moe.moe_gemm_bf16(A, W, D, trans_a=ta, trans_w=tw, workspace=workspace(M, N, K))
    a, w = f64(A), f64(W)
    check(D.contiguous(), a.T if ta else a, w.T if tw else w, None, "none", False, None)
