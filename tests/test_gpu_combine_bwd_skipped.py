"""Skipped slots of the combine's gradient next to Inf and NaN: dweights is 0 for a slot whose output_index names no row,
whatever the token's dZ holds, and what the other slots and tokens get does not change."""

import pytest
import torch

import int4_weights_amd as moe
from gpu_helpers import DEV, require_gpu

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _run(dz, y, oi, w, dy=True):
    T, k = oi.shape
    ws = torch.full((max(16, moe.moe_unpermute_combine_bwd_workspace_bytes(T, k, y.shape[0])),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    dY = torch.full_like(y, 3.0) if dy else None
    dW = torch.full((T, k), 9.0, device=DEV)
    moe.moe_unpermute_combine_bwd(dz, y, oi, w if dy else None, dY, dW, workspace=ws)
    torch.cuda.synchronize()
    return dY, dW


# 1024, 512 and 256 threads, 2, 4 and 8 slots a workgroup; the last three with the row table in the workspace
@pytest.mark.parametrize("T,k,N", [(5, 1, 8), (30, 8, 2056), (90, 8, 72), (300, 8, 1032), (300, 6, 264), (600, 8, 64),
                                   (700, 6, 2056), (2100, 2, 24)])
@pytest.mark.parametrize("dy", [True, False])
def test_zero_whatever_dz_holds(T, k, N, dy):
    require_gpu()
    g = torch.Generator().manual_seed(T + k)
    rows = T * k + 5
    dz = torch.randn(T, N, generator=g).to(torch.bfloat16)
    y = torch.randn(rows, N, generator=g).to(torch.bfloat16).to(DEV)
    oi = torch.randperm(rows, generator=g)[:T * k].view(T, k).to(torch.int32)
    w = torch.rand(T, k, generator=g).to(DEV)
    oi[0] = -1  # a padded token: no slot names a row, its dZ was never written
    oi[2, k // 2] = rows  # past the end
    oi[T - 1, 0] = -7
    bad = dz.clone()
    bad[0] = NAN
    bad[2, N - 1] = INF
    bad[T - 1, 0], bad[T - 1, N // 2] = -INF, NAN
    skip = ((oi < 0) | (oi >= rows)).to(DEV)
    hurt = torch.zeros(T, dtype=torch.bool, device=DEV)
    hurt[[0, 2, T - 1]] = True
    cY, cW = _run(dz.to(DEV), y, oi.to(DEV), w, dy)
    dY, dW = _run(bad.to(DEV), y, oi.to(DEV), w, dy)
    assert (dW[skip] == 0).all()
    assert torch.equal(dW[~hurt], cW[~hurt])
    assert not torch.isfinite(dW[hurt[:, None] & ~skip]).any()  # a named row's sum holds the Inf or NaN
    if dy:
        named = oi.to(DEV)[hurt[:, None] & ~skip].long()
        keep = torch.ones(rows, dtype=torch.bool, device=DEV)
        keep[named] = False
        assert torch.equal(dY[keep], cY[keep])


def test_dropped_route_leaves_the_router_gradient_finite():
    """A route that a full expert dropped keeps its topk_id: its weight's gradient reaches moe_router_topk_bwd as 0."""
    require_gpu()
    T, E, k, N = 9, 16, 4, 64
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(T, E, generator=g).to(DEV)
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    moe.moe_router_topk(logits, ids, w)
    oi = torch.arange(T * k, dtype=torch.int32).view(T, k)
    oi[4] = -1  # all four dropped
    dz = torch.randn(T, N, generator=g).to(torch.bfloat16)
    dz[4] = NAN
    y = torch.randn(T * k, N, generator=g).to(torch.bfloat16).to(DEV)
    _, dw = _run(dz.to(DEV), y, oi.to(DEV), w)
    dl = torch.full_like(logits, 5.0)
    moe.moe_router_topk_bwd(logits, ids, dw, dl)
    torch.cuda.synchronize()
    assert torch.isfinite(dl).all() and (dl[4] == 0).all()
