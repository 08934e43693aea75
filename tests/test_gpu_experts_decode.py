"""moe_experts_decode against the float64 oracle: every format, order and row-block size; skipped, repeated and foreign
experts; residuals in place; device status; limits; streams and graphs."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu, u16

pytestmark = pytest.mark.gpu


class Layer:
    """Weights of a format, row-major and packed, and the values they stand for."""

    def __init__(self, fmt, E, H, I, seed=0, std=0.1):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.E, self.H, self.I = fmt, E, H, I
        self.w, self.s, self.wp, self.sp, self.val = {}, {}, {}, {}, {}
        for name, (N, K) in {"13": (2 * I, H), "2": (H, I)}.items():
            w = (torch.randn(E, N, K, generator=g) * std).to(torch.bfloat16).to(DEV)
            if fmt == "bf16":
                q, s, p, sp = w, None, torch.empty_like(w), None
                moe.moe_pack_weight_bf16(q, p)
                val = w.double().cpu().numpy()
            elif fmt == "fp8":
                q, s = torch.empty(E, N, K, dtype=torch.uint8, device=DEV), torch.empty(E, N // 128, K // 128, device=DEV)
                moe.moe_quant_weight_fp8(w, q, s)
                s *= torch.rand(s.shape, generator=g).add(0.5).to(DEV)  # no powers of two
                p, sp = torch.empty_like(q), s
                moe.moe_pack_weight_fp8(q, p)
                big = s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
                val = (q.view(torch.float8_e4m3fn).double() * big).cpu().numpy()
            elif fmt == "fp4":
                q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
                s = torch.empty(E, N, K // 32, dtype=torch.uint8, device=DEV)
                w = (w.view(E, N, -1, 32) * torch.exp2(torch.randint(-3, 4, (E, N, K // 32, 1), generator=g)).to(DEV)).view(E, N, K)
                moe.moe_quant_weight_fp4(w.to(torch.bfloat16), q, s)  # scales that differ from block to block
                p, sp = torch.empty_like(q), torch.empty_like(s)
                moe.moe_pack_weight_fp4(q, s, p, sp)
                codes = torch.stack((q & 15, q >> 4), -1).view(E, N, K).cpu().numpy()
                val = oracle.e2m1_decode_table()[codes] * np.repeat(np.exp2(s.double().cpu().numpy() - 127), 32, 2)
            else:
                q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
                s = torch.empty(E, N, K // 128, dtype=torch.float16, device=DEV)
                moe.moe_quant_weight_int4(w, q, s)
                p, sp = torch.empty_like(q), torch.empty_like(s)
                moe.moe_pack_weight_int4(q, s, p, sp)
                codes = torch.stack((q & 15, q >> 4), -1).view(E, N, K).double() - 8
                val = (codes * s.double().repeat_interleave(128, 2)).cpu().numpy()
            self.w[name], self.s[name], self.wp[name], self.sp[name], self.val[name] = q, s, p, sp, val

    def run(self, x, ids, p, z=None, packed=False, residual=None, status=None, ws=None, stream=None):
        z = torch.empty_like(x) if z is None else z
        w, s = (self.wp, self.sp) if packed else (self.w, self.s)
        if ws is None:
            ws = torch.empty(max(16, moe.moe_experts_decode_workspace_bytes(*ids.shape, self.I)), dtype=torch.uint8, device=DEV)
        moe.moe_experts_decode(x, ids, p, w["13"], w["2"], z, weights=self.fmt, s13=s["13"], s2=s["2"], packed=packed,
                               residual=residual, dev_status=status, workspace=ws, stream=stream)
        return z


def inputs(T, k, E, H, seed, dropped=0, one=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32) if k <= E else \
        torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if one:
        ids[:] = E - 1
    ids.view(-1)[torch.randperm(T * k, generator=g)[:dropped]] = -1
    return x, ids.to(DEV), torch.softmax(torch.randn(T, k, generator=g), 1).to(DEV)


def check(L, z, x, ids, p, residual=None):
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    # h and Z are rounded to bf16 (half a step: 2^-8); sums of up to H (I) products in fp32, scaled block sums among them, are
    # off by at most 2 * terms * 2^-24 of the products' magnitudes; 4-bit codes are added up around an offset of 136: 128 + q
    # (at most 143) and 136 in place of q - 8
    extra = 279.0 * max(float(L.s[n].float().abs().max()) for n in ("13", "2")) if L.fmt == "int4" else 0.0
    acc = 2.0 * max(L.H, L.I) * 2.0 ** -24
    ref, bound = oracle.experts_decode(f(x), f(ids), f(p), L.val["13"], L.val["2"], None if residual is None else f(residual),
                                       rounding=2.0 ** -8 * (1 + 2.0 ** -8), accumulation=acc, w_extra=extra)
    err = np.abs(f(z) - ref)
    assert np.isfinite(f(z)).all()
    assert (err <= bound + 2.0 ** -8 * (np.abs(ref) + bound) + 1e-30).all(), float((err - bound).max())
    # the two roundings are independent, each well under half a step on average
    n = np.linalg.norm(ref)
    assert n == 0 or np.linalg.norm(f(z) - ref) < 2.0 ** -8 * n


SHAPES = [  # T, k, E, H, I, dropped, one expert for all
    (1, 1, 1, 128, 128, 0, False),
    (1, 8, 16, 512, 256, 0, False),
    (2, 3, 5, 640, 384, 1, False),
    (3, 2, 64, 256, 128, 0, False),
    (7, 4, 6, 384, 256, 5, False),
    (16, 2, 4, 256, 640, 0, False),
    (5, 1, 3, 1152, 128, 0, True),
    (37, 3, 4, 256, 128, 0, True),     # 111 rows of one expert
    (61, 8, 12, 256, 256, 3, False),
    (128, 8, 9, 128, 128, 0, False),   # the most tokens and routes
    (64, 16, 40, 128, 128, 17, False),
    (1, 64, 2, 128, 256, 0, False),    # one token, the same experts many times
    (9, 8, 200, 4224, 128, 0, False),  # more than 256 column blocks
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4", "fp4"])
@pytest.mark.parametrize("T,k,E,H,I,dropped,one", SHAPES)
def test_against_the_oracle(fmt, packed, T, k, E, H, I, dropped, one):
    require_gpu()
    E = min(E, 12) if H > 2000 else E
    L = Layer(fmt, E, H, I, seed=T + k)
    x, ids, p = inputs(T, k, E, H, T * k + E, dropped, one)
    res = torch.randn(T, H, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).to(DEV) if (T + k) % 2 else None
    check(L, L.run(x, ids, p, packed=packed, residual=res), x, ids, p, res)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4", "fp4"])
def test_orders_agree_and_results_repeat(fmt):
    """Packed weights are the same numbers; nothing depends on timing.  (The orders add a block's products up differently, so
    they agree to the sums' rounding only: at most a step of bf16.)"""
    require_gpu()
    L = Layer(fmt, 10, 512, 384)
    x, ids, p = inputs(19, 4, 10, 512, 3)
    a = L.run(x, ids, p)
    for _ in range(5):
        assert torch.equal(a, L.run(x, ids, p))
    b = L.run(x, ids, p, packed=True)
    assert torch.equal(b, L.run(x, ids, p, packed=True))
    check(L, b, x, ids, p)


def test_skipped_slots_and_status():
    require_gpu()
    L = Layer("fp8", 6, 256, 128)
    x, ids, p = inputs(4, 3, 6, 256, 1)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids[1, :] = -1          # nothing for this token
    ids[2, 1] = -2147483648
    z = L.run(x, ids, p, status=status)
    assert int(status) == 0 and (z[1] == 0).all()
    check(L, z, x, ids, p)
    res = torch.randn_like(x)
    z = L.run(x, ids, p, residual=res)
    assert torch.equal(z[1], res[1])
    ids[0, 0], ids[3, 2] = 6, 2147483647
    z = L.run(x, ids, p, status=status)
    assert int(status) == moe.DEV_ID_RANGE
    check(L, z, x, ids, p)
    L.run(x, ids, p)  # not reported
    ids[:] = -1
    assert (L.run(x, ids, p) == 0).all()
    assert torch.equal(L.run(x, ids, p, residual=res), res)


def test_weights_of_skipped_slots_do_not_count():
    """A skipped slot's weight and an inactive expert's weights may be anything."""
    require_gpu()
    L = Layer("bf16", 5, 256, 128)
    x, ids, p = inputs(6, 2, 4, 256, 2)
    ids[3, 1] = -1
    z = L.run(x, ids, p)
    p[3, 1] = float("nan")
    L.w["13"][4].fill_(float("nan"))
    L.w["2"][4].fill_(float("inf"))
    assert torch.equal(z, L.run(x, ids, p))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "int4", "fp4"])
def test_a_bad_row_stays_alone(fmt):
    """Infinities and NaN of one token reach no other, whatever rows share its matrix instructions."""
    require_gpu()
    L = Layer(fmt, 3, 256, 128)
    x, ids, p = inputs(11, 2, 3, 256, 4)
    z = L.run(x, ids, p)
    x2 = x.clone()
    x2[5] = float("nan")
    x2[8, 17] = float("inf")
    y = L.run(x2, ids, p)
    keep = [t for t in range(11) if t not in (5, 8)]
    assert torch.equal(y[keep], z[keep])
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[8]).all()


def test_residual_in_place_and_untouched_neighbours():
    require_gpu()
    L = Layer("int4", 8, 384, 256)
    x, ids, p = inputs(5, 2, 8, 384, 6)
    room = torch.full((7, 384), 3.0, dtype=torch.bfloat16, device=DEV)
    res = torch.randn(5, 384, device=DEV).to(torch.bfloat16)
    want = L.run(x, ids, p, residual=res)
    room[1:6] = res
    L.run(x, ids, p, z=room[1:6], residual=room[1:6])
    assert torch.equal(room[1:6], want) and (room[0] == 3).all() and (room[6] == 3).all()
    x2 = x.clone()
    L.run(x2, ids, p, z=x2, residual=res)  # over the input
    assert torch.equal(x2, want)
    ws = torch.full((moe.moe_experts_decode_workspace_bytes(5, 2, 256) + 64,), 77, dtype=torch.uint8, device=DEV)
    L.run(x, ids, p, ws=ws[:-64])
    assert (ws[-64:] == 77).all()


def test_no_tokens():
    require_gpu()
    L = Layer("bf16", 2, 128, 128)
    x, ids, p = (torch.empty(0, 128, dtype=torch.bfloat16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV),
                 torch.empty(0, 2, device=DEV))
    moe.moe_experts_decode(x, ids, p, L.w["13"], L.w["2"], torch.empty_like(x), weights="bf16")


def test_streams_and_graph():
    """Two calls at once on two streams with workspaces of their own; captured, replayed with new inputs in place."""
    require_gpu()
    A, B = Layer("fp8", 8, 512, 256, 1), Layer("int4", 8, 512, 256, 2)
    (xa, ia, pa), (xb, ib, pb) = inputs(9, 4, 8, 512, 1), inputs(17, 3, 8, 512, 2)
    za, zb = A.run(xa, ia, pa), B.run(xb, ib, pb, packed=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = (torch.empty(moe.moe_experts_decode_workspace_bytes(*i.shape, 256), dtype=torch.uint8, device=DEV) for i in (ia, ib))
    outs = []
    for _ in range(8):
        oa, ob = torch.empty_like(xa), torch.empty_like(xb)
        torch.cuda.synchronize()
        A.run(xa, ia, pa, z=oa, ws=wa, stream=s1)
        B.run(xb, ib, pb, z=ob, ws=wb, packed=True, stream=s2)
        outs.append((oa, ob))
    torch.cuda.synchronize()
    assert all(torch.equal(a, za) and torch.equal(b, zb) for a, b in outs)
    g = torch.cuda.CUDAGraph()
    z = torch.empty_like(xa)
    with torch.cuda.graph(g):
        A.run(xa, ia, pa, z=z, ws=wa)
    for i in range(4):
        x2, i2, p2 = inputs(9, 4, 8, 512, 10 + i, dropped=i)
        want = A.run(x2, i2, p2)
        xa.copy_(x2), ia.copy_(i2), pa.copy_(p2)
        z.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want)


def test_experts_past_32_bits():
    """An expert whose weights lie beyond 2^32 bytes."""
    require_gpu()
    E, H, I = 1024, 2048, 1024
    w13 = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device=DEV)
    w2 = torch.zeros(E, H, I, dtype=torch.uint8, device=DEV)
    s13, s2 = torch.ones(E, 2 * I // 128, H // 128, device=DEV), torch.ones(E, H // 128, I // 128, device=DEV)
    L = Layer("fp8", 1, H, I, 5)
    for n, w, s in (("13", w13, s13), ("2", w2, s2)):
        w[E - 1], s[E - 1] = L.w[n][0], L.s[n][0]
    x, ids, p = inputs(2, 1, 1, H, 8)
    want = L.run(x, ids, p)
    z = torch.empty_like(x)
    ws = torch.empty(moe.moe_experts_decode_workspace_bytes(2, 1, I), dtype=torch.uint8, device=DEV)
    moe.moe_experts_decode(x, torch.full_like(ids, E - 1), p, w13, w2, z, weights="fp8", s13=s13, s2=s2, workspace=ws)
    assert torch.equal(z, want)
