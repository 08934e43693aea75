"""moe_experts_decode against the float64 oracle at sizes that reach every kernel of every format (test_decode_plan.py says which), and
with routes that crowd on a few of many experts."""

import pytest
import torch

import int4_weights_amd as moe
from decode_shapes import FORMATS, REACHED
from gpu_helpers import DEV, require_gpu
from test_gpu_experts_decode import Layer, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,shape", [(f, s) for f in FORMATS for s in REACHED[f]], ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_every_kernel(fmt, shape):
    require_gpu()
    T, k, E, H, I = shape
    L = Layer(fmt, E, H, I, seed=T + E)
    x, ids, p = inputs(T, k, E, H, T * k + E, dropped=T // 9)
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(DEV) if T % 2 else None
    n = moe.moe_experts_decode_workspace_bytes(T, k, I)
    ws = torch.full((n + 256,), 77, dtype=torch.uint8, device=DEV)
    for packed in (False, True):
        z = L.run(x, ids, p, packed=packed, residual=res, ws=ws[:n])
        check(L, z, x, ids, p, res)
        assert torch.equal(z, L.run(x, ids, p, packed=packed, residual=res)) and (ws[n:] == 77).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,k,E,H", [(37, 8, 200, 128), (61, 8, 130, 256), (128, 8, 1000, 128), (20, 3, 70, 4224)])
def test_crowded_experts(fmt, T, k, E, H):
    """Experts by Zipf's law: a few with many times the mean, so many jobs each, most with none; a token's experts may repeat."""
    require_gpu()
    L = Layer(fmt, E, H, 128, seed=E)
    x, ids, p = inputs(T, k, E, H, T)
    g = torch.Generator().manual_seed(T)
    order = torch.randperm(E, generator=g)
    ids = order[torch.multinomial(1 / (1 + torch.arange(E).float()), T * k, replacement=True, generator=g)].view(T, k).to(torch.int32).to(DEV)
    assert int(torch.bincount(ids.view(-1).long()).max()) > 8  # rows of the largest job at these means
    for packed in (False, True):
        check(L, L.run(x, ids, p, packed=packed), x, ids, p)
