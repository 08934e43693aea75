"""MoeDecodeLayer: how long a forward's result lasts, with and without a z of the caller's."""

import pytest
import torch

from gpu_helpers import DEV, require_gpu
from int4_weights_amd.layer import MoeDecodeLayer
from test_gpu_experts_decode import Layer, check, inputs

pytestmark = pytest.mark.gpu


def test_a_result_in_the_callers_z_outlives_the_next_forward():
    require_gpu()
    L = Layer("fp8", 6, 256, 128)
    layer = MoeDecodeLayer(L.w["13"], L.w["2"], 2, 9, "fp8", L.s["13"], L.s["2"])
    steps = [inputs(T, 2, 6, 256, T) for T in (9, 4, 7)]
    kept = [layer.forward(x, ids, p, z=torch.empty_like(x)) for x, ids, p in steps]
    own = [layer.forward(x, ids, p) for x, ids, p in steps]
    for z, (x, ids, p) in zip(kept, steps):
        check(L, z, x, ids, p)
    assert torch.equal(own[-1], kept[-1])                       # the layer's buffer holds the last one
    assert all(z.data_ptr() == layer.Z.data_ptr() for z in own)
    h = kept[0].clone()
    layer.forward(kept[0], steps[0][1], steps[0][2], z=kept[0], residual=h)  # a layer's output as the next one's input, in place
    check(L, kept[0], h, steps[0][1], steps[0][2], h)
