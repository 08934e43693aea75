"""Two choices of one MoeRouter alive at once: the second forward before the first one's gradient."""

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from int4_weights_amd.layer import MoeRouter

pytestmark = pytest.mark.gpu

E, K, T = 64, 6, 40


def _data(seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, E, generator=g).to(DEV), torch.randn(T, K, generator=g).to(DEV)


def _own():
    return torch.empty(T, K, dtype=torch.int32, device=DEV), torch.empty(T, K, device=DEV)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_two_forwards_before_the_first_gradient(score):
    require_gpu()
    (a, ga), (b, gb) = _data(1), _data(2)
    r = MoeRouter(E, K, T, score=score)
    want = []
    for x, gx in ((a, ga), (b, gb)):  # one batch after the other
        ids, w = r.forward(x)
        want.append((ids.clone(), w.clone(), r.backward(x, ids, gx, torch.empty_like(x)).clone()))
    ia, wa = r.forward(a, *_own())
    ib, wb = r.forward(b, *_own())
    da = r.backward(a, ia, ga, torch.empty_like(a))
    db = r.backward(b, ib, gb, torch.empty_like(b))
    torch.cuda.synchronize()
    for got, ref in zip(((ia, wa, da), (ib, wb, db)), want):
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_own_buffers_may_be_longer_than_the_routers():
    require_gpu()
    x, _ = _data(3)
    r = MoeRouter(E, K, 3)
    ids, w = _own()
    got = r.forward(x, ids, w)
    assert got[0] is ids and got[1] is w
    big = MoeRouter(E, K, T).forward(x)
    torch.cuda.synchronize()
    assert torch.equal(ids, big[0]) and torch.equal(w, big[1])


def test_refusals():
    require_gpu()
    x, _ = _data(4)
    r = MoeRouter(E, K, T)
    ids, w = _own()
    with pytest.raises(ValueError):
        r.forward(x, ids)  # one of the two
    with pytest.raises(ValueError):
        r.forward(x, None, w)
    with pytest.raises(ValueError):
        r.forward(x, ids[:3], w[:3])
    with pytest.raises(ValueError):
        r.forward(x, ids[:, :3].contiguous(), w[:, :3].contiguous())  # another top-k than the router's
    with pytest.raises(ValueError):
        MoeRouter(E, K, 3).forward(x)  # more tokens than its buffers hold
