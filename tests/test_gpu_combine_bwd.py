"""The combine's gradient on the GPU against the float64 oracle.

dY of a row named once is one fp32 product rounded to bf16: half a bf16 step (2^-8) plus 2^-24, relative.  A row named
by c slots: c roundings of the running sum more.  dweights: a sum of N products, each fused with the running sum: at
most N * 2^-24 of the sum of magnitudes (the lanes' partial sums only shorten the chains).
"""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _run(dz, y, oi, w, dy=True, dw=True):
    T, k = oi.shape
    ws = torch.empty(max(16, moe.moe_unpermute_combine_bwd_workspace_bytes(T, k, y.shape[0])), dtype=torch.uint8, device=DEV)
    ws.fill_(0xA5)
    dY = torch.full_like(y, 3.0) if dy else None
    dW = torch.full((T, k), float("nan"), device=DEV) if dw else None
    moe.moe_unpermute_combine_bwd(dz, y if dw else None, oi, w if dy else None, dY, dW, workspace=ws)
    torch.cuda.synchronize()
    return dY, dW


def _check(dz, y, oi, w):
    dY, dW = _run(dz, y, oi, w)
    o, N = oi.cpu().numpy(), y.shape[1]
    ry, named, rw = oracle.combine_bwd(_f64(dz), _f64(y), o, _f64(w))
    my, _, mw = oracle.combine_bwd(np.abs(_f64(dz)), np.abs(_f64(y)), o, np.abs(_f64(w)))
    got = _f64(dY)
    assert (got[~named] == 3.0).all(), "rows that no slot names were written"
    cnt = np.bincount(o[(o >= 0) & (o < y.shape[0])], minlength=y.shape[0])[:, None]
    assert (np.abs(got - ry)[named] <= (2.0 ** -8 * np.abs(ry) + (cnt + 1) * U * my * 1.01 + 1e-38)[named]).all()
    assert (np.abs(_f64(dW) - rw) <= N * U * mw + 1e-38).all()
    skip = (o < 0) | (o >= y.shape[0])
    assert (_f64(dW)[skip] == 0).all()
    return dY, dW


def _inputs(T, k, N, rows, seed, unique=True):
    g = torch.Generator().manual_seed(seed)
    dz = torch.randn(T, N, generator=g).to(torch.bfloat16).to(DEV)
    y = torch.randn(rows, N, generator=g).to(torch.bfloat16).to(DEV)
    if unique:
        oi = torch.randperm(rows, generator=g)[:T * k].view(T, k).to(torch.int32)
    else:
        oi = torch.randint(-2, rows + 2, (T, k), generator=g).to(torch.int32)
    return dz, y, oi, torch.rand(T, k, generator=g).to(DEV)


@pytest.mark.parametrize("T,k,N,rows", [
    (1, 1, 8, 1), (1, 8, 7168, 8), (5, 3, 2056, 40), (61, 8, 520, 500), (3, 64, 136, 200), (7, 9, 4096, 70),
    (513, 8, 64, 4200),  # more than 4096 routes: the workspace path
    (700, 6, 8, 4300), (4097, 1, 16, 4097),
    (130, 8, 4104, 1100), (300, 7, 1032, 2200), (450, 5, 2056, 2300), (300, 13, 264, 4000), (1500, 3, 72, 4600),
])
def test_against_oracle(T, k, N, rows):
    require_gpu()
    dz, y, oi, w = _inputs(T, k, N, rows, T + N)
    oi[0, 0] = -1
    if T > 2:
        oi[2, k // 2] = rows  # past the end: skipped
    _check(dz, y, oi.to(DEV), w)


@pytest.mark.parametrize("T,k,N,rows", [(6, 4, 24, 9), (40, 8, 2064, 12), (600, 8, 16, 1500), (5000, 1, 8, 3)])
def test_rows_named_several_times(T, k, N, rows):
    require_gpu()
    dz, y, oi, w = _inputs(T, k, N, rows, T, unique=False)
    a = _check(dz, y, oi.to(DEV), w)
    b = _run(dz, y, oi.to(DEV), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,k,N,rows", [(30, 8, 8216, 200), (1030, 4, 2072, 3000)])
def test_rows_named_several_times_wide(T, k, N, rows):
    """Rows wider than one turn of a workgroup's threads."""
    require_gpu()
    dz, y, oi, w = _inputs(T, k, N, rows, T, unique=False)
    _check(dz, y, oi.to(DEV), w)


def test_many_rows_named_twice():
    """Half a million routes, every row named by two of them far apart."""
    require_gpu()
    T, k, N = 65536, 8, 8
    g = torch.Generator().manual_seed(1)
    rows = T * k // 2
    oi = torch.cat([torch.randperm(rows, generator=g), torch.randperm(rows, generator=g)]).view(T, k)
    dz = torch.randn(T, N, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.rand(T, k, generator=g).to(DEV)
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    dY, _ = _run(dz, y, oi.to(torch.int32).to(DEV), w)
    v = (w.double()[:, :, None] * dz.double()[:, None]).view(-1, N)
    at = oi.view(-1).to(DEV)
    ref = torch.zeros(rows, N, dtype=torch.float64, device=DEV).index_add_(0, at, v)
    mag = torch.zeros_like(ref).index_add_(0, at, v.abs())
    assert ((dY.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 3 * U * 1.01 * mag + 1e-38).all()


@pytest.mark.parametrize("T", [50, 600])
def test_outputs_alone(T):
    require_gpu()
    dz, y, oi, w = _inputs(T, 8, 128, 8 * T + 3, T)
    oi = oi.to(DEV)
    dY, dW = _run(dz, y, oi, w)
    assert torch.equal(_run(dz, y, oi, w, dw=False)[0], dY)
    assert torch.equal(_run(dz, y, oi, w, dy=False)[1], dW)


def test_empty_and_refusals():
    require_gpu()
    z = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    y = torch.ones(5, 64, dtype=torch.bfloat16, device=DEV)
    oi = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    dy = y.clone()
    moe.moe_unpermute_combine_bwd(z, y, oi, w, dy, w.clone())
    assert torch.equal(dy, y)
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    dz = torch.ones(3, 64, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((3, 2), 9.0, device=DEV)
    moe.moe_unpermute_combine_bwd(dz, y[:0], none, torch.ones(3, 2, device=DEV), y[:0].clone(), dw)
    assert (dw == 0).all()
    with pytest.raises(ValueError):
        moe.moe_unpermute_combine_bwd(dz, y, none, None, dy, dw)
    with pytest.raises(ValueError):
        moe.moe_unpermute_combine_bwd(dz, None, none, torch.ones(3, 2, device=DEV), dy, dw)
    with pytest.raises(ValueError):
        moe.moe_unpermute_combine_bwd(dz, y, none, torch.ones(3, 2, device=DEV), dy[:4].contiguous(), dw)
    big = torch.zeros(5000, 1, dtype=torch.int32, device=DEV)
    with pytest.raises(moe.MoeError):
        moe.moe_unpermute_combine_bwd(torch.ones(5000, 64, dtype=torch.bfloat16, device=DEV), y, big,
                                      torch.ones(5000, 1, device=DEV), dy, torch.ones(5000, 1, device=DEV))
