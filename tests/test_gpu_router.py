"""The router and its gradient on the GPU against the float64 oracle.

Choice: equal (keys are ordered as their 64-bit values).  Weights and gradients: fp32 roundings counted in units of
2^-24 of the value.  A score is an exponential (the hardware exp2's ulp is 2 units, its argument's low part and the
product 2, the rounded difference x - m one per unit of |x - m|), a sum 1 + exp (1) and a quotient (1); a weight has
two of those and the sum over the slots or the row (6 levels across the lanes, up to 32 values in one), and the
scale (1).  2 * (|x - m| + 6) + 38 + 2 units are rounded up to 64 + 2 |x - m|.
"""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _run(x, k, ids_fill=-9, **kw):
    T = x.shape[0]
    ids = torch.full((T, k), ids_fill, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    moe.moe_router_topk(x, ids, w, **kw)
    torch.cuda.synchronize()
    return ids, w


def _check(x, k, **kw):
    ids, w = _run(x, k, **kw)
    x64 = x.detach().float().cpu().numpy().astype(np.float64)
    okw = dict(kw)
    if okw.get("bias") is not None:
        okw["bias"] = okw["bias"].cpu().numpy()
    ri, rw = oracle.router_topk(x64, k, **okw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    sel = np.where(ri >= 0, np.take_along_axis(x64, np.maximum(ri, 0), 1), 0.0)
    span = np.zeros(x.shape[0])
    fin = np.where(np.isfinite(x64), x64, np.nan)
    if np.isfinite(x64).any():
        with np.errstate(all="ignore"):
            span = np.nan_to_num(np.nanmax(fin, 1)) + np.abs(np.where(np.isfinite(sel), sel, 0)).max(1)
    err = np.abs(w.cpu().numpy().astype(np.float64) - rw)
    assert (err <= U * (64 + 2 * np.abs(span)[:, None]) * np.abs(rw) + 1e-37).all()
    return ids, w


SHAPES = [  # T, E, k, groups, kept, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 5, 5, 1, 1, 1), (16, 128, 8, 1, 1, 1), (7, 60, 4, 6, 3, 2),
    (65, 256, 8, 8, 4, 2), (33, 257, 9, 1, 1, 1), (9, 1000, 64, 1, 1, 1), (5, 1024, 64, 64, 4, 2), (6, 990, 7, 33, 5, 1),
    (130, 64, 6, 8, 3, 1), (17, 160, 6, 8, 3, 1), (4, 24, 3, 24, 3, 2), (2, 512, 1, 2, 1, 2),
]


@pytest.mark.parametrize("T,E,k,G,TG,gt", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_choice_and_weights(T, E, k, G, TG, gt, score, bias):
    require_gpu()
    g = torch.Generator().manual_seed(T * E + k)
    for dt in (torch.float32, torch.bfloat16):
        x = (torch.randn(T, E, generator=g) * 2).to(dt).to(DEV)
        b = (torch.randn(E, generator=g) * 0.1).to(DEV) if bias else None
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            _check(x, k, score=score, bias=b, n_group=G, topk_group=TG, group_top=gt, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_expert(score):
    require_gpu()
    x = torch.zeros(4, 256, device=DEV)
    x[1, 100] = 1.0
    x[2, ::2] = -0.0  # equal to +0
    x[3] = torch.arange(256, device=DEV) // 32  # groups of equal logits
    for b in (None, torch.zeros(256, device=DEV), torch.full((256,), -3.0, device=DEV)):
        for G, TG, gt in ((1, 1, 1), (8, 4, 1), (8, 4, 2)):
            _check(x, 8, score=score, bias=b, n_group=G, topk_group=TG, group_top=gt)


def test_keys_closer_than_fp32_are_ordered_exactly():
    """Pairs of experts whose scores plus bias differ by far less than an fp32 ulp, in both index orders, and
    groups whose sums do."""
    require_gpu()
    rng = np.random.default_rng(5)
    T, E = 64, 64
    x = np.sort(rng.standard_normal((T, E)), 1).astype(np.float32)
    # bias cancels the scores of row 0 up to its fp32 rounding: every key of row 0 is about 1 + 1e-8
    s = 1 / (1 + np.exp(-x[0].astype(np.float64)))
    b = (1.0 - s).astype(np.float32)
    x[1:] = x[0]  # the same near-ties, with the experts' values nudged by single ulps
    for t in range(1, T):
        e = rng.integers(0, E, 8)
        x[t, e] = np.nextafter(x[t, e], np.float32(10 if t % 2 else -10))
    xt, bt = torch.from_numpy(x).to(DEV), torch.from_numpy(b).to(DEV)
    for G, TG, gt in ((1, 1, 1), (8, 4, 2), (8, 2, 1)):
        _check(xt, 8, score="sigmoid", bias=bt, n_group=G, topk_group=TG, group_top=gt)
    p = np.exp(x[0].astype(np.float64) - x[0].max())
    b = (0.5 - p / p.sum()).astype(np.float32)
    _check(xt, 8, score="softmax", bias=torch.from_numpy(b).to(DEV), n_group=8, topk_group=3, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_unavailable_experts(score, bias):
    require_gpu()
    g = torch.Generator().manual_seed(1)
    x = torch.randn(12, 40, generator=g)
    x[0] = float("-inf")
    x[1] = float("nan")
    x[2, 3:] = float("-inf")            # fewer than k left
    x[3, :20] = float("nan")            # whole groups empty
    x[4, torch.randperm(40, generator=g)[:35]] = float("-inf")
    x[5, 7] = torch.finfo(torch.float32).min
    x[6] = torch.finfo(torch.float32).min
    x[7, ::3] = float("-inf")
    x[8, 5] = 80.0
    x[9] -= 60.0                        # scores far below 1, renormalised without underflow
    b = torch.randn(40, generator=g) * 0.2 if bias else None
    if bias:
        b[11] = float("-inf")           # out for every token
        b[12] = float("nan")
        b = b.to(DEV)
    for G, TG, gt in ((1, 1, 1), (4, 2, 1), (8, 4, 2), (20, 5, 2)):
        ids, w = _check(x.to(DEV), 8, score=score, bias=b, n_group=G, topk_group=TG, group_top=gt)
        assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[1] == -1).all() and (w[1] == 0).all()
        if bias:
            assert not ((ids == 11) | (ids == 12)).any()


def test_infinite_logits():
    require_gpu()
    x = torch.zeros(2, 16, device=DEV)
    x[0, 5] = float("inf")
    x[1, 3] = x[1, 9] = float("inf")
    ids, w = _run(x, 4)
    assert ids.cpu().tolist() == [[5, 0, 1, 2], [3, 9, 0, 1]]
    assert w.cpu().tolist() == [[1, 0, 0, 0], [0.5, 0.5, 0, 0]]
    ids, w = _run(x, 2, score="sigmoid", renormalize=False)
    assert ids.cpu().tolist() == [[5, 0], [3, 9]] and w.cpu().tolist() == [[1, 0.5], [1, 1]]


def test_strided_rows_and_offsets():
    require_gpu()
    big = torch.randn(50, 333, device=DEV)
    for dt in (torch.float32, torch.bfloat16):
        v = big.to(dt)[:, 1:257]  # a row start that no vector load fits
        a = _check(v, 8, score="sigmoid")
        b = _run(v.contiguous(), 8, score="sigmoid")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _bwd(x, ids, dw, **kw):
    d = torch.full_like(x, float("nan"))
    moe.moe_router_topk_bwd(x, ids, dw, d, **kw)
    torch.cuda.synchronize()
    return d


def _check_bwd(x, ids, dw, score, renormalize, scale):
    d = _bwd(x, ids, dw, score=score, renormalize=renormalize, scale=scale).float().cpu().numpy().astype(np.float64)
    x64 = x.float().cpu().numpy().astype(np.float64)
    i, g = ids.cpu().numpy(), dw.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        ref = oracle.router_topk_bwd(x64, i, g, score, renormalize, scale)
    # every summand's magnitude: the same formula with |g|, and the mean's part added rather than subtracted
    w = oracle.router_weights(x64, i, score, renormalize, 1.0)
    mean = (np.abs(g) * w).sum(1) * abs(scale)
    mag = np.zeros_like(ref)
    for t in range(x.shape[0]):
        for r, e in enumerate(i[t]):
            if 0 <= e < x.shape[1] and x64[t, e] > -np.inf:
                mag[t, e] += w[t, r] * (abs(scale * g[t, r]) + (mean[t] if renormalize else 0.0))
        if score == "softmax" and not renormalize:
            mag[t] += oracle.router_scores(x64[t], "softmax") * mean[t]
    fin = np.where(np.isfinite(x64), x64, 0.0)
    units = 128 + 4 * (fin.max(1) - fin.min(1))[:, None]  # two weights' errors, the sums, as above
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0
    assert (np.abs(d - ref) <= U * units * mag + half * np.abs(ref) + 1e-37).all()
    assert (d[mag == 0] == 0).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 256, 8), (64, 128, 8), (9, 1000, 64), (3, 1024, 13), (130, 37, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient(T, E, k, score, renorm):
    require_gpu()
    g = torch.Generator().manual_seed(T + E)
    for dt in (torch.float32, torch.bfloat16):
        x = (torch.randn(T, E, generator=g) * 2).to(dt).to(DEV)
        ids, _ = _run(x, k, score=score)
        dw = torch.randn(T, k, generator=g).to(DEV)
        _check_bwd(x, ids, dw, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_unusual_slots(score, renorm):
    """Empty slots, ids out of range, one expert in several slots, unavailable experts, a row without any."""
    require_gpu()
    g = torch.Generator().manual_seed(3)
    x = torch.randn(8, 70, generator=g)
    ids = torch.stack([torch.randperm(70, generator=g)[:6] for _ in range(8)]).to(torch.int32)
    ids[0] = -1
    ids[1, 2:] = -1
    ids[2, 1] = 70
    ids[2, 4] = 1 << 30
    ids[3] = 5
    ids[4, 3] = ids[4, 0]
    x[5, ids[5, 0].item()] = float("-inf")
    x[5, ids[5, 1].item()] = float("nan")
    x[6] = float("-inf")
    x[7] -= 70.0
    dw = torch.randn(8, 6, generator=g)
    dw[0] = float("nan")  # of empty slots: not read into anything
    _check_bwd(x.to(DEV), ids.to(DEV), torch.nan_to_num(dw).to(DEV), score, renorm, 1.5)
    d = _bwd(x.to(DEV), ids.to(DEV), dw.to(DEV), score=score, renormalize=renorm)
    assert (d[0] == 0).all()


def test_gradient_against_differences():
    require_gpu()
    g = torch.Generator().manual_seed(9)
    x = torch.randn(3, 24, generator=g, dtype=torch.float64)
    ids, _ = _run(x.float().to(DEV), 4, score="sigmoid")
    x = x.float().double()  # the values the GPU sees
    dw = torch.randn(3, 4, generator=g)
    d = _bwd(x.float().to(DEV), ids, dw.to(DEV), score="sigmoid", scale=2.5).cpu().double().numpy()
    i, h = ids.cpu().numpy(), 1e-5
    for t in range(3):
        for e in range(24):
            p, m = x.clone(), x.clone()
            p[t, e] += h
            m[t, e] -= h
            num = (dw.double().numpy() * (oracle.router_weights(p.numpy(), i, "sigmoid", True, 2.5)
                                          - oracle.router_weights(m.numpy(), i, "sigmoid", True, 2.5))).sum() / (2 * h)
            # differences are good to h^2 and 1e-16 / h, fp32 to a few units of values below 4
            assert abs(num - d[t, e]) < 2e-6


def test_gradient_strided():
    require_gpu()
    x = torch.randn(20, 99, device=DEV)[:, 3:80]
    ids, _ = _run(x, 5)
    dw = torch.randn(20, 5, device=DEV)
    out = torch.full((20, 90), 7.0, device=DEV)
    moe.moe_router_topk_bwd(x, ids, dw, out[:, 2:79], renormalize=False)
    ref = _bwd(x.contiguous(), ids, dw, renormalize=False)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 2:79], ref)
    assert (out[:, :2] == 7).all() and (out[:, 79:] == 7).all()


def test_refusals_of_the_binding():
    require_gpu()
    x = torch.randn(4, 16, device=DEV)
    i = torch.empty(4, 2, dtype=torch.int32, device=DEV)
    w = torch.empty(4, 2, device=DEV)
    for bad in (dict(score="relu"), dict(bias=torch.zeros(15, device=DEV)), dict(bias=torch.zeros(16, device=DEV).double())):
        with pytest.raises(ValueError):
            moe.moe_router_topk(x, i, w, **bad)
    with pytest.raises(ValueError):
        moe.moe_router_topk(x.t(), i, w)
    with pytest.raises(ValueError):
        moe.moe_router_topk(x.half(), i, w)
    with pytest.raises(moe.MoeError):
        moe.moe_router_topk(x, i, w, n_group=3)
    with pytest.raises(moe.MoeError):
        moe.moe_router_topk(x[:1].expand(4, 16), i, w)  # rows on top of one another
    with pytest.raises(ValueError):
        moe.moe_router_topk_bwd(x, i, w, x.to(torch.bfloat16))
