"""The new calls as they are used together: a decode step (gate projection, router, experts, shared expert added to them) and a
training step of a dense layer (forward, gradients accumulated over micro-batches), against the oracle, captured and replayed."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, fp8_quant_weight_gpu, require_gpu
from int4_weights_amd.layer import DenseFP8Linear, DenseLinear, MoeDecodeLayer, MoeFP8Layer, MoeRouter

pytestmark = pytest.mark.gpu

E, H, I, K, T = 16, 512, 256, 4, 23


def f64(t):
    return t.double().cpu().numpy()


def bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


class Step:
    """One decode step of a layer with routed FP8 experts and a shared one in bf16."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.q13, self.s13 = fp8_quant_weight_gpu(bf(g, E, 2 * I, H, scale=0.05))
        self.q2, self.s2 = fp8_quant_weight_gpu(bf(g, E, H, I, scale=0.05))
        self.gate = DenseLinear(bf(g, E, H, scale=0.2))
        self.router = MoeRouter(E, K, T, score="sigmoid", bias=(torch.randn(E, generator=g) * 0.1).to(DEV), n_group=4,
                                topk_group=2, group_top=2, scale=2.5)
        self.experts = MoeDecodeLayer(self.q13, self.q2, K, T, s13=self.s13, s2=self.s2)
        self.up = DenseLinear(bf(g, 2 * I, H, scale=0.05), act="silu", gated=True)
        self.down = DenseLinear(bf(g, H, I, scale=0.05))
        self.x = bf(g, T, H)
        self.logits = torch.empty(T, E, device=DEV)
        self.h, self.y = (torch.empty(T, n, dtype=torch.bfloat16, device=DEV) for n in (I, H))

    def run(self):
        self.gate.forward(self.x, self.logits)
        ids, w = self.router.forward(self.logits)
        z = self.experts.forward(self.x, ids, w, residual=self.x)
        self.up.forward(self.x, self.h)
        self.down.forward(self.h, self.y, residual=z)
        return self.logits, ids, w, z, self.h, self.y


def close(got, ref, steps=2.0):
    """Within `steps` half steps of bf16 of the value, and of a hundredth of the largest (sums that cancel)."""
    d = np.abs(f64(got) - ref)
    return (d <= steps * 2.0 ** -8 * (np.abs(ref) + 0.05 * np.abs(ref).max())).all()


def test_decode_step_against_the_oracle():
    require_gpu()
    s = Step()
    logits, ids, w, z, h, y = (t.clone() for t in s.run())
    torch.cuda.synchronize()
    x = f64(s.x)
    ref, _, mag = oracle.linear(x, f64(s.gate.w))
    assert (np.abs(f64(logits) - ref) <= 2 * H * 2.0 ** -24 * mag).all()
    ri, rw = oracle.router_topk(f64(logits), K, "sigmoid", s.router.bias.cpu().numpy(), 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), ri) and np.allclose(f64(w), rw, rtol=1e-5)
    val = [oracle.e4m3_decode_table()[q.cpu().numpy()] * np.repeat(np.repeat(f64(sc), 128, 1), 128, 2)
           for q, sc in ((s.q13, s.s13), (s.q2, s.s2))]
    ref, bound = oracle.experts_decode(x, ri, f64(w), *val, residual=x, rounding=2.0 ** -8, accumulation=2 * H * 2.0 ** -24)
    assert (np.abs(f64(z) - ref) <= bound + 2.0 ** -8 * (np.abs(ref) + bound)).all()
    ref, _, _ = oracle.linear(x, f64(s.up.w), None, "silu", True)
    assert close(h, ref)
    ref, _, _ = oracle.linear(f64(h), f64(s.down.w), residual=f64(z))
    assert close(y, ref)
    assert int(s.experts.dev_status) == 0


def test_the_grouped_path_gives_the_same_layer():
    """The decode kernels against the packed FP8 path of the same weights, whose activations are quantised to E4M3 twice: half a
    step of E4M3 is 2^-4 of a value, and the errors of a sum's terms are independent."""
    require_gpu()
    s = Step(3)
    _, ids, w, _, _, _ = s.run()
    z = s.experts.forward(s.x, ids, w)
    up = MoeFP8Layer(s.q13, s.s13, K, T)
    up.quant_route(s.x, ids)
    q = torch.empty(up.rows_cap, I, dtype=torch.uint8, device=DEV)
    sf = torch.empty(up.rows_cap, I // 128, device=DEV)
    up.gemm_swiglu(q, sf)
    D = torch.empty(up.rows_cap, H, dtype=torch.bfloat16, device=DEV)
    up.gemm(q, sf, D, s.q2, s.s2, H, I)
    zg = up.combine(w, D, torch.empty(T, H, dtype=torch.bfloat16, device=DEV))
    a, b = f64(z), f64(zg)
    assert np.linalg.norm(a - b) < 2.0 ** -4 * np.linalg.norm(a)


def test_decode_step_captured_and_replayed():
    require_gpu()
    s = Step(1)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = s.run()
    other = Step(2)
    for i in range(4):
        s.x.copy_(bf(torch.Generator().manual_seed(20 + i), T, H))
        want = [t.clone() for t in s.run()]
        for t in captured:
            t.view(torch.uint8).fill_(0x21)
        other.run()  # the program's own work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_decode_layer_refuses_what_does_not_fit():
    require_gpu()
    s = Step(4)
    with pytest.raises(ValueError, match="room for"):
        s.experts.forward(torch.zeros(T + 1, H, dtype=torch.bfloat16, device=DEV), None, None)
    with pytest.raises(ValueError, match="at most"):
        MoeDecodeLayer(s.q13, s.q2, K, moe.DECODE_MAX_TOKENS + 1, s13=s.s13, s2=s.s2)


class Train:
    """A dense layer (SwiGLU up with bias, down with a residual) and the gradients of everything it reads."""

    def __init__(self, seed, tokens):
        g = torch.Generator().manual_seed(seed)
        self.x, self.dz = bf(g, tokens, H), bf(g, tokens, H)
        self.up = DenseLinear(bf(g, 2 * I, H, scale=0.06), (torch.randn(2 * I, generator=g) * 0.1).to(DEV), "silu", True)
        self.down = DenseLinear(bf(g, H, I, scale=0.06))
        n = lambda *sh: torch.empty(*sh, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        self.pre, self.h, self.z, self.dh, self.dp, self.dx = (n(tokens, c) for c in (2 * I, I, H, I, 2 * I, H))
        self.dw1, self.dw2, self.db = (torch.zeros(*sh, device=DEV) for sh in ((2 * I, H), (H, I), (2 * I,)))

    def run(self):
        self.up.forward(self.x, self.h, pre=self.pre)
        self.down.forward(self.h, self.z, residual=self.x)
        self.down.grad_weight(self.dz, self.h, self.dw2)
        self.down.grad_input(self.dz, self.dh)
        self.up.grad_pre(self.dh, self.pre, self.dp, self.db)
        self.up.grad_weight(self.dp, self.x, self.dw1)
        self.up.grad_input(self.dp, self.dx, residual=self.dz)
        return self.z, self.dx, self.dw1, self.dw2, self.db

    def reference(self):
        """Every call's formula in 64 bits, on the operands that it got."""
        x, dz, w1, w2, b = (f64(t) for t in (self.x, self.dz, self.up.w, self.down.w, self.up.bias))
        h, _, _ = oracle.linear(x, w1, b, "silu", True)
        dp = oracle.act_bwd(f64(self.dh), f64(self.pre), "silu", True)
        return {"h": (self.h, h), "z": (self.z, f64(self.h) @ w2.T + x), "dh": (self.dh, dz @ w2), "dp": (self.dp, dp),
                "dx": (self.dx, f64(self.dp) @ w1 + dz)}, \
            {"dw2": (self.dw2, dz.T @ f64(self.h)), "dw1": (self.dw1, f64(self.dp).T @ x), "db": (self.db, dp.sum(0))}


@pytest.mark.parametrize("tokens", [1, 37, 333, 1500])
def test_training_step_against_the_oracle(tokens):
    require_gpu()
    s = Train(1, tokens)
    s.run()
    torch.cuda.synchronize()
    rounded, summed = s.reference()
    for name, (got, ref) in rounded.items():
        assert close(got, ref), name
    for name, (got, ref) in summed.items():  # fp32: sums of up to `tokens` terms
        assert np.linalg.norm(f64(got) - ref) <= 2 * (tokens + 8) * 2.0 ** -24 * np.linalg.norm(ref) + 1e-30, name
    # the chain's own gradient, whose intermediates are not rounded: five roundings of bf16 (pre, h, dh, dP, dx), each at most 2^-8
    # of its values and on average less than half of that, independent from term to term
    x, dz, w1, w2, b = (f64(t) for t in (s.x, s.dz, s.up.w, s.down.w, s.up.bias))
    _, pre, _ = oracle.linear(x, w1, b, "silu", True)
    dp = oracle.act_bwd(dz @ w2, pre, "silu", True)
    for got, ref in ((s.dx, dp @ w1 + dz), (s.dw1, dp.T @ x), (s.db, dp.sum(0))):
        assert np.linalg.norm(f64(got) - ref) < 5 * 2.0 ** -8 * np.linalg.norm(ref)


def test_micro_batches_accumulate():
    require_gpu()
    a = Train(5, 200)
    a.run()
    once = [t.clone() for t in (a.dw1, a.dw2, a.db)]
    a.run()
    for t, o in zip((a.dw1, a.dw2, a.db), once):
        assert (t - 2 * o).abs().max() <= 2 * 210 * 2.0 ** -24 * 2 * o.abs().max() + 1e-30


def test_training_step_captured_and_replayed():
    require_gpu()
    s, other = Train(6, 333), Train(7, 100)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = s.run()
    for i in range(4):
        s.x.copy_(bf(torch.Generator().manual_seed(30 + i), 333, H))
        for t in (s.dw1, s.dw2, s.db):
            t.zero_()
        want = [t.clone() for t in s.run()]
        for t in captured:
            t.zero_()
        other.run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_bf16_and_fp8_shared_experts_agree():
    """DenseLinear beside DenseFP8Linear: the same weights, codes against values; x quantised to E4M3, half a step 2^-4."""
    require_gpu()
    g = torch.Generator().manual_seed(8)
    w, x = bf(g, 384, H, scale=0.05), bf(g, 70, H)
    q, sc = fp8_quant_weight_gpu(w[None])
    val = (q[0].view(torch.float8_e4m3fn).float() * sc[0].repeat_interleave(128, 0).repeat_interleave(128, 1)).to(torch.bfloat16)
    y, z = (torch.empty(70, 384, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    DenseFP8Linear(q[0], sc[0], 70).forward(x, y)
    DenseLinear(val).forward(x, z)
    assert np.linalg.norm(f64(y) - f64(z)) < 2.0 ** -4 * np.linalg.norm(f64(z))
