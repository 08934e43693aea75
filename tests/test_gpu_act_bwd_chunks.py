"""moe_act_bwd past 1024 rows, where the rows are cut into chunks and a second launch adds the chunks' lines: accumulating, strided, in place,
bad values, guarded workspaces, two streams, captured and replayed."""

import pytest
import torch

import int4_weights_amd as moe
from gpu_helpers import DEV, require_gpu
from test_gpu_act_bwd import check, f64, inputs, run

pytestmark = pytest.mark.gpu
SHAPES = [(1025, 34), (1501, 1042), (2047, 64), (4099, 1034)]  # odd rows, columns that end inside a lane's 8


def scratch(M, N):
    n = moe.moe_act_bwd_workspace_bytes(M, N)
    assert n > 0  # several chunks
    return n


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act,gated", [("none", False), ("gelu", False), ("silu", True)])
def test_accumulated_in_a_guarded_workspace(shape, act, gated):
    require_gpu()
    M, N = shape
    n = scratch(M, N)
    dD, pre = inputs(M, N, gated, M)
    before = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(DEV)
    room = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    dP, db = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), before.clone()
    moe.moe_act_bwd(dD, pre, dP, dbias=db, act=act, gated=gated, accumulate=True, workspace=room[:n])
    check(dP, db, dD, pre, act, gated, f64(before))
    assert (room[n:] == 0xA5).all()
    alone = torch.empty_like(db)
    run(dD, pre, act, gated, dP=None, dbias=alone)
    assert torch.equal(db, before + alone)  # one addition, of the same sums
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_act_bwd(dD, pre, dP, dbias=db, act=act, gated=gated, workspace=room[:n - 16])


@pytest.mark.parametrize("gated", [False, True])
def test_strided_and_in_place(gated):
    require_gpu()
    M, N = 1501, 1042
    scratch(M, N)
    dD, pre = inputs(M, N, gated, 4)
    wb = torch.empty(N, device=DEV)
    want = run(dD, pre, "gelu", gated, dbias=wb)
    check(want, wb, dD, pre, "gelu", gated)
    h = dD.shape[1]
    a, b, c = (torch.full((M, w + 3 * i), 5.0, dtype=torch.bfloat16, device=DEV) for i, w in ((1, h), (2, N), (3, N)))
    a[:, :h], b[:, :N] = dD, pre
    db = torch.empty_like(wb)
    ws = torch.empty(scratch(M, N), dtype=torch.uint8, device=DEV)
    moe.moe_act_bwd(a[:, :h], b[:, :N], c[:, :N], dbias=db, act="gelu", gated=gated, workspace=ws)
    assert torch.equal(c[:, :N], want) and (c[:, N:] == 5).all() and torch.equal(db, wb)
    p = pre.clone()
    run(dD, p, "gelu", gated, dP=p, dbias=db)  # over the pre-activation
    assert torch.equal(p, want) and torch.equal(db, wb)
    if not gated:
        d = dD.clone()
        run(d, pre, "gelu", gated, dP=d, dbias=db)
        assert torch.equal(d, want) and torch.equal(db, wb)


def test_a_bad_value_stays_in_its_column():
    require_gpu()
    M, N = 1501, 1042
    dD, pre = inputs(M, N, False, 5)
    db, db2 = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    dP = run(dD, pre, "silu", False, dbias=db)
    dD[1200, 9] = float("nan")
    pre[1500, 1041] = float("inf")
    dP2 = run(dD, pre, "silu", False, dbias=db2)
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[[9, 1041]] = False
    assert torch.equal(db[keep], db2[keep]) and not torch.isfinite(db2[~keep]).any() and torch.equal(dP[:, keep], dP2[:, keep])
    assert torch.isnan(dP2[1200, 9]) and torch.equal(dP[:1200], dP2[:1200])


def test_two_streams_and_graph():
    require_gpu()
    M, N = 1501, 1042
    n = scratch(M, N)
    dD, pre = inputs(M, N, True, 6)
    d2, p2 = inputs(M, N, False, 7)
    db, db2 = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    a, b = run(dD, pre, "silu", True, dbias=db), run(d2, p2, "relu", False, dbias=db2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    w1, w2 = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(n, dtype=torch.uint8, device=DEV)
    outs = [[torch.empty_like(t) for t in (a, db, b, db2)] for _ in range(6)]
    torch.cuda.synchronize()
    for oa, oda, ob, odb in outs:
        moe.moe_act_bwd(dD, pre, oa, dbias=oda, act="silu", gated=True, workspace=w1, stream=s1)
        moe.moe_act_bwd(d2, p2, ob, dbias=odb, act="relu", workspace=w2, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o in outs for x, y in zip(o, (a, db, b, db2)))
    out, acc = torch.empty_like(a), torch.zeros(N, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_act_bwd(dD, pre, out, dbias=acc, act="silu", gated=True, accumulate=True, workspace=w1)
    acc.zero_()
    total = torch.zeros_like(acc)
    for i in range(4):  # a captured step adds to the gradient of the steps before
        x, y = inputs(M, N, True, 10 + i)
        dD.copy_(x), pre.copy_(y)
        want = run(x, y, "silu", True, dbias=total, accumulate=True)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(acc, total)
