"""moe_experts_decode with MXFP4 scales over the whole of E8M0, where code times scale lies past bf16's range or below its normal
numbers: activations of the other extreme bring the products back to ordinary size."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu
from test_gpu_experts_decode import Layer, check, inputs

pytestmark = pytest.mark.gpu


class Scaled(Layer):
    """Random codes under given scale bytes: s13 [E, 2I, H/32], s2 [E, H, I/32]."""

    def __init__(self, s13, s2, seed):
        g = torch.Generator().manual_seed(seed)
        self.fmt = "fp4"
        self.E, self.H, self.I = s2.shape[0], s2.shape[1], s13.shape[1] // 2
        self.w, self.s, self.wp, self.sp, self.val = {}, {}, {}, {}, {}
        for name, s in (("13", s13), ("2", s2)):
            E, N, K = s.shape[0], s.shape[1], 32 * s.shape[2]
            q = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
            codes = torch.stack((q & 15, q >> 4), -1).view(E, N, K).numpy()
            val = oracle.e2m1_decode_table()[codes] * np.repeat(np.exp2(s.double().numpy() - 127), 32, 2)
            q, s = q.to(DEV), s.to(torch.uint8).to(DEV)
            p, sp = torch.empty_like(q), torch.empty_like(s)
            moe.moe_pack_weight_fp4(q, s, p, sp)
            self.w[name], self.s[name], self.wp[name], self.sp[name], self.val[name] = q, s, p, sp, val


def full(value, *shape):
    return torch.full(shape, int(value))


def steps(seed, T, e):
    """Values of magnitude 1 to 1.75 times 2^e (e per column): normal bf16 numbers from e = -126 on."""
    g = torch.Generator().manual_seed(seed)
    v = 1 + torch.randint(0, 4, (T, e.numel()), generator=g).double() / 4
    v = torch.where(torch.rand(v.shape, generator=g) < 0.5, -v, v) * torch.exp2(e.double())
    return v.to(torch.bfloat16).to(DEV)


E, H, I, T, K = 2, 256, 128, 5, 2
BYTES = [0, 1, 2, 3, 127, 251, 252, 253, 254]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("byte", BYTES)
def test_up_projection(byte, packed):
    """Codes of 0.5 to 6 times 2^(byte - 127) against activations of about 2^(125 - byte)."""
    require_gpu()
    L = Scaled(full(byte, E, 2 * I, H // 32), full(120, E, H, I // 32), byte)
    _, ids, p = inputs(T, K, E, H, 1)
    x = steps(2, T, full(min(max(125 - byte, -126), 124), H))
    check(L, L.run(x, ids, p, packed=packed), x, ids, p)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("byte", BYTES)
def test_down_projection(byte, packed):
    """The same for h, which the up rows' scales bring to about 2^(127 - byte) (not below 2^-100)."""
    require_gpu()
    e = min(max(127 - byte, -100), 118)
    s13 = full(121, E, 2 * I, H // 32)
    s13[:, I:] = 121 + e
    L = Scaled(s13, full(byte, E, H, I // 32), byte)
    x, ids, p = inputs(T, K, E, H, 3)
    check(L, L.run(x, ids, p, packed=packed), x, ids, p)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,K", [(1, 1), (T, K), (23, 2), (60, 2)])  # 4, 8 and 16 rows a job
def test_scales_that_differ(T, K, packed):
    """Blocks of every size side by side, rows of weights up to 8 times apart."""
    require_gpu()
    g = torch.Generator().manual_seed(T)

    def mixed(n, k):
        base = torch.tensor([254, 1, 253, 127, 60, 252, 200, 4])[torch.randperm(max(8, k // 32), generator=g) % 8][:k // 32]
        return base, (base - torch.randint(0, 4, (E, n, k // 32), generator=g)).clamp(0, 254)

    b13, s13 = mixed(2 * I, H)
    _, s2 = mixed(H, I)
    L = Scaled(s13, full(124, E, H, I // 32), T)
    _, ids, p = inputs(T, K, E, H, 5)
    x = steps(6, T, (125 - b13).clamp(-126, 124).repeat_interleave(32))
    check(L, L.run(x, ids, p, packed=packed), x, ids, p)
    b = torch.tensor([253, 3, 252, 127])  # of h's four blocks, whose up rows make up for it
    s13 = full(121, E, 2 * I, H // 32)
    s13[:, I:] = 121 + (127 - b).clamp(-100, 100).repeat_interleave(32)[None, :, None]
    L = Scaled(s13, (b - torch.randint(0, 4, (E, H, I // 32), generator=g)).clamp(0, 254), T + 1)
    x, ids, p = inputs(T, K, E, H, 7)
    check(L, L.run(x, ids, p, packed=packed), x, ids, p)


def test_quantised_weights_at_the_end_of_bf16():
    """moe_quant_weight_fp4 writes scale 2^126 and codes of 4 for the largest bf16 numbers."""
    require_gpu()
    L = Scaled(full(127, E, 2 * I, H // 32), full(120, E, H, I // 32), 1)
    w = ((torch.rand(E, 2 * I, H, generator=torch.Generator().manual_seed(2)) * 2 - 1) * 3.35e38).to(torch.bfloat16).to(DEV)
    q, s = L.w["13"], L.s["13"]
    moe.moe_quant_weight_fp4(w, q, s)
    assert int(s.max()) == 253 and bool(((q & 7) == 6).any())
    codes = torch.stack((q & 15, q >> 4), -1).view(E, 2 * I, H).cpu().numpy()
    L.val["13"] = oracle.e2m1_decode_table()[codes] * np.repeat(np.exp2(s.double().cpu().numpy() - 127), 32, 2)
    moe.moe_pack_weight_fp4(q, s, L.wp["13"], L.sp["13"])
    _, ids, p = inputs(T, K, E, H, 1)
    x = steps(2, T, full(-126, H))
    for packed in (False, True):
        check(L, L.run(x, ids, p, packed=packed), x, ids, p)


@pytest.mark.parametrize("packed", [False, True])
def test_a_nan_scale(packed):
    """Scale byte 255 is E8M0's NaN: it reaches the results that its block is part of, and no others."""
    require_gpu()
    T, E = 6, 3
    x, ids, p = inputs(T, 1, E, H, 9)
    ids[:, 0] = torch.arange(T, device=DEV) % E
    s13, s2 = full(124, E, 2 * I, H // 32), full(124, E, H, I // 32)
    want = Scaled(s13, s2, 4).run(x, ids, p, packed=packed)
    s13[1, I + 70, 5], s2[2, 33, 1] = 255, 255
    got = Scaled(s13, s2, 4).run(x, ids, p, packed=packed)
    bad = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    bad[ids[:, 0] == 1] = True                       # one h of expert 1 goes into every column
    bad[(ids[:, 0] == 2).nonzero()[:, 0], 33] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
