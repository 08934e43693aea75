"""The new calls as they are used together: router -> experts -> combine, a shared expert beside them, and the way back;
captured into graphs; on a stream of their own; with shared workspaces; at offsets past 32 bits."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, fp8_quant_weight_gpu, require_gpu, u16
from int4_weights_amd.layer import DenseFP8Linear, MoeFP8Layer, MoeRouter

pytestmark = pytest.mark.gpu

T, E, K, N, TOPK = 200, 16, 512, 384, 4


def _f64(t):
    return t.double().cpu().numpy()


def _bf(*shape, g, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


class Step:
    """One training step of a router, its experts' forward, a shared expert and their gradients."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.x, self.dz = _bf(T, K, g=g), _bf(T, N, g=g)
        self.logits = torch.randn(T, E, generator=g).to(DEV)
        w, ws = _bf(E, N, K, g=g, scale=0.05), _bf(N, K, g=g, scale=0.05)
        self.wq, self.wsf = fp8_quant_weight_gpu(w)
        sq, ssf = fp8_quant_weight_gpu(ws[None])
        tq, tsf = fp8_quant_weight_gpu(ws.t().contiguous()[None])
        self.router = MoeRouter(E, TOPK, T, score="sigmoid", bias=(torch.randn(E, generator=g) * 0.1).to(DEV), n_group=4,
                                topk_group=2, group_top=2, scale=2.5)
        self.layer = MoeFP8Layer(self.wq, self.wsf, TOPK, T)
        self.shared = DenseFP8Linear(sq[0], ssf[0], T, tq[0], tsf[0])
        self.y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        self.dD = torch.zeros_like(self.layer.D)
        self.dw = torch.empty(T, TOPK, device=DEV)
        self.dlogits = torch.empty_like(self.logits)
        self.dx = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
        self.gw = torch.zeros(N, K, device=DEV)

    def run(self):
        self.ids, self.tw = self.router.forward(self.logits)
        self.z = self.layer.forward(self.x, self.ids, self.tw, fused_quant=True)
        self.shared.forward(self.x, self.y)
        self.layer.combine_backward(self.dz, self.tw, self.dD, self.dw)
        self.router.backward(self.logits, self.ids, self.dw, self.dlogits)
        self.shared.grad_input(self.dz, self.dx)
        self.shared.grad_weight(self.dz, self.x, self.gw, accumulate=False)
        return [t.clone() for t in (self.ids, self.tw, self.z, self.y, self.dD, self.dw, self.dlogits, self.dx, self.gw)]


def test_step_against_the_oracle():
    require_gpu()
    s = Step()
    ids, tw, z, y, dD, dw, dl, dx, gw = s.run()
    torch.cuda.synchronize()
    ri, rw = oracle.router_topk(_f64(s.logits), TOPK, "sigmoid", s.router.bias.cpu().numpy(), 4, 2, 2, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert np.allclose(_f64(tw), rw, rtol=2.0 ** -24 * 100)
    # forward: the experts' product of the quantised operands, combined with the router's weights
    xq, xs = oracle.quant_act(u16(s.x))
    ref = np.zeros((T, N))
    rows = np.zeros((T, TOPK, N))
    for e in range(E):
        t, r = np.nonzero(ri == e)
        rows[t, r] = oracle.dense_gemm_fp8(xq[t], xs[t], s.wq[e].cpu().numpy(), s.wsf[e].cpu().numpy())[0]
    ref = (rw[:, :, None] * rows).sum(1)
    assert oracle.calc_diff(_f64(z), ref) < 1e-3 and oracle.elementwise_ok(_f64(z), ref)
    # backward through the combine and the router, from the GPU's own packed rows
    D = s.layer.D
    oi = s.layer.output_index.cpu().numpy()
    ry, named, rdw = oracle.combine_bwd(_f64(s.dz), np.nan_to_num(_f64(D)), oi, _f64(tw))
    assert (np.abs(_f64(dD) - ry)[named] <= 2.0 ** -7 * np.abs(ry)[named] + 1e-30).all()
    assert np.allclose(_f64(dw), rdw, rtol=1e-4, atol=1e-4 * np.abs(rdw).max())
    rdl = oracle.router_topk_bwd(_f64(s.logits), ri, _f64(dw), "sigmoid", True, 2.5)
    assert np.allclose(_f64(dl), rdl, rtol=1e-4, atol=1e-5 * np.abs(rdl).max())
    # the shared expert's three products
    ref = oracle.dense_gemm_fp8(xq, xs, s.shared.w.cpu().numpy(), s.shared.sfw.cpu().numpy())[0]
    assert oracle.elementwise_ok(_f64(y), ref)
    yq, ys = oracle.quant_act(u16(s.dz))
    ref = oracle.dense_gemm_fp8(yq, ys, s.shared.wt.cpu().numpy(), s.shared.sfwt.cpu().numpy())[0]
    assert oracle.elementwise_ok(_f64(dx), ref)
    a, sa = oracle.quant_act_t(u16(s.dz))
    b, sb = oracle.quant_act_t(u16(s.x))
    ref, mag = oracle.dense_gemm_fp8(a, sa, b, sb, 1)
    assert (np.abs(_f64(gw) - ref) <= 300 * 2.0 ** -24 * mag).all()
    # and the quantised gradient is the gradient: E4M3's half step of either operand, 2 * 2^-4 per product
    true = _f64(s.dz).T @ _f64(s.x)
    assert np.linalg.norm(_f64(gw) - true) < 2 * 2.0 ** -4 * np.linalg.norm(true)


def test_gradient_of_the_weights_against_differences():
    """d loss / d logits through combine and router against central differences of the float64 chain."""
    require_gpu()
    s = Step(3)
    ids, tw, z, y, dD, dw, dl, *_ = s.run()
    torch.cuda.synchronize()
    oi, i = s.layer.output_index.cpu().numpy(), ids.cpu().numpy()
    Y, dz, x = np.nan_to_num(_f64(s.layer.D)), _f64(s.dz), _f64(s.logits)

    def loss(v, t):
        w = oracle.router_weights(v, i[t:t + 1], "sigmoid", True, 2.5)
        return float((oracle.combine(Y, oi[t:t + 1], w) * dz[t]).sum())

    for t in (0, 57, 199):
        for e in range(E):
            p, m = x[t:t + 1].copy(), x[t:t + 1].copy()
            p[0, e] += 1e-5
            m[0, e] -= 1e-5
            num = (loss(p, t) - loss(m, t)) / 2e-5
            assert abs(num - _f64(dl)[t, e]) < 1e-4 * max(1.0, np.abs(_f64(dw)[t]).max())


def test_captured_and_replayed():
    require_gpu()
    s = Step(1)
    eager = s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = s.run()
    for i in range(4):
        for t in captured:
            t.view(torch.uint8).fill_(0x11 * (i + 1))
        s.dD.zero_()
        other = Step(2 + i % 2).run()  # the program's own work between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        del other


def test_two_graphs_share_a_workspace():
    """Split K, captured twice with one workspace, replayed in turn."""
    require_gpu()
    gen = torch.Generator().manual_seed(4)
    M, n, k = 131, 256, 7168
    need = moe.moe_gemm_fp8_workspace_bytes(M, n, k)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    ops, graphs, outs, refs = [], [], [], []
    for _ in range(2):
        a = torch.randint(0, 120, (M, k), generator=gen).to(torch.uint8).to(DEV)
        w = torch.randint(0, 120, (n, k), generator=gen).to(torch.uint8).to(DEV)
        sa, sw = torch.rand(M, k // 128, generator=gen).to(DEV), torch.rand(n // 128, k // 128, generator=gen).to(DEV)
        d = torch.empty(M, n, dtype=torch.bfloat16, device=DEV)
        ops.append((a, sa, w, sw, d))
        moe.moe_gemm_fp8(a, sa, w, sw, d, workspace=ws)
        refs.append(d.clone())
    torch.cuda.synchronize()
    for op in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_gemm_fp8(*op, workspace=ws)
        graphs.append(g)
        outs.append(op[4])
    for i in range(6):
        outs[i % 2].zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], refs[i % 2])
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])


@pytest.mark.parametrize("t,fill", [(1100, 0xFF), (1100, 0x00), (5000, 0xFF)])
def test_combine_gradient_with_workspace_in_graphs(t, fill):
    """Past 4096 routes: two graphs that share a workspace of any content; padded tokens (id -1) in the batch."""
    require_gpu()
    gen = torch.Generator().manual_seed(t)
    n, rows = 256, t * TOPK + 40
    need = moe.moe_unpermute_combine_bwd_workspace_bytes(t, TOPK, rows)
    assert need > 0
    ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
    sets = []
    for _ in range(2):
        oi = torch.randperm(rows, generator=gen)[:t * TOPK].view(t, TOPK).to(torch.int32)
        oi[-100:] = -1
        y, dz = _bf(rows, n, g=gen), _bf(t, n, g=gen)
        w = torch.rand(t, TOPK, generator=gen).to(DEV)
        dY, dw = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV), torch.empty(t, TOPK, device=DEV)
        want = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV)
        on = oi[:-100].reshape(-1).long().to(DEV)
        want[on] = (w[:-100, :, None] * dz[:-100, None].float()).to(torch.bfloat16).view(-1, n)
        sets.append((dz, y, oi.to(DEV), w, dY, dw, want))
    graphs = []
    for dz, y, oi, w, dY, dw, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_unpermute_combine_bwd(dz, y, oi, w, dY, dw, workspace=ws)
        graphs.append(g)
    first = [None, None]
    for i in range(6):
        dz, y, oi, w, dY, dw, want = sets[i % 2]
        dY.fill_(7.0)
        dw.fill_(5.0)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(dY, want)
        assert not dw[-100:].any()
        first[i % 2] = dw.clone() if first[i % 2] is None else first[i % 2]
        assert torch.equal(dw, first[i % 2])
        s = Step(7).run()  # the program's own work between replays
        del s


def test_two_streams_at_once():
    """Two split-K products and two gradients in flight together, each with a workspace of its own."""
    require_gpu()
    a, b = Step(8), Step(9)
    ra, rb = a.run(), b.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            ga = a.run()
        with torch.cuda.stream(s2):
            gb = b.run()
        torch.cuda.synchronize()
        for x, y in zip(ra + rb, ga + gb):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_layer_refusals_and_empty_batches():
    require_gpu()
    s = Step(10)
    with pytest.raises(ValueError):
        s.shared.forward(torch.zeros(T + 1, K, dtype=torch.bfloat16, device=DEV), s.y)
    with pytest.raises(ValueError):
        s.shared.forward(torch.zeros(3, N, dtype=torch.bfloat16, device=DEV), s.y[:3])
    with pytest.raises(ValueError):
        DenseFP8Linear(s.shared.w, s.shared.sfw, T).grad_input(s.dz, s.dx)
    none = torch.zeros(0, K, dtype=torch.bfloat16, device=DEV)
    s.shared.forward(none, s.y[:0])
    s.gw.fill_(2.0)
    assert (s.shared.grad_weight(s.dz[:0], none, s.gw) == 2).all()
    assert not s.shared.grad_weight(s.dz[:0], none, s.gw, accumulate=False).any()


def test_on_another_stream():
    require_gpu()
    s = Step(5)
    ref = s.run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = s.run()
    # and by argument
    logits = s.logits.clone()
    ids, w = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_router_topk(logits, ids, w, score="sigmoid", bias=s.router.bias, n_group=4, topk_group=2, group_top=2,
                        scale=2.5, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1])


def test_repeated_calls_are_bit_identical():
    require_gpu()
    s = Step(6)
    first = s.run()
    for _ in range(5):
        for a, b in zip(first, s.run()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------------------- offsets past 32 bits --
def test_long_combine_gradient():
    """Rows of Y past 2^31 elements."""
    require_gpu()
    n, rows, t = 4096, 540000, 64
    y = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    dY = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(1)
    oi = (rows - 1 - torch.randperm(600, generator=g)[:t * 2]).view(t, 2).to(torch.int32)
    at = oi.view(-1).long().to(DEV)
    y[at] = torch.randn(t * 2, n, generator=g).to(torch.bfloat16).to(DEV)
    dz, w = torch.randn(t, n, generator=g).to(torch.bfloat16).to(DEV), torch.rand(t, 2, generator=g).to(DEV)
    dw = torch.empty(t, 2, device=DEV)
    moe.moe_unpermute_combine_bwd(dz, y, oi.to(DEV), w, dY, dw)
    torch.cuda.synchronize()
    ref = (y[at].double().view(t, 2, n) * dz.double()[:, None]).sum(2)
    assert torch.allclose(dw.double(), ref, rtol=1e-4, atol=1e-3)
    want = (w[:, :, None] * dz.float()[:, None]).to(torch.bfloat16).view(-1, n)
    assert torch.equal(dY[at], want)
    dY[at] = 0
    assert not dY.any()


def test_long_product_output_and_operands():
    """D past 2^31 elements, A past 2^31 bytes (row strides wider than the rows)."""
    require_gpu()
    M, n, k, lda, ldd = 70000, 64, 128, 33024, 33000
    big = torch.zeros(M, lda, dtype=torch.uint8, device=DEV)
    out = torch.zeros(M, ldd, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(2)
    codes = torch.tensor([0x00, 0x38, 0xB8, 0x40], dtype=torch.uint8)
    a = codes[torch.randint(0, 4, (M, k), generator=g)].to(DEV)
    w = codes[torch.randint(0, 4, (n, k), generator=g)].to(DEV)
    big[:, :k] = a
    sa, sw = torch.ones(M, 1, device=DEV), torch.full((1, 1), 0.5, device=DEV)
    moe.moe_gemm_fp8(big[:, :k], sa, w, sw, out[:, :n])
    torch.cuda.synchronize()
    ref = (a.view(torch.float8_e4m3fn).float() @ w.view(torch.float8_e4m3fn).float().t()) * 0.5
    assert torch.equal(out[:, :n], ref.to(torch.bfloat16))  # whole and half numbers: exact before the one rounding
    assert not out[:, n:n + 64].any()


def test_long_router_and_quantiser():
    require_gpu()
    rows = (1 << 31) // 512 + 300  # logits past 2^31 elements, strided
    x = torch.zeros(rows, 512, dtype=torch.bfloat16, device=DEV)
    x[-7:, :64] = torch.randn(7, 64, device=DEV).to(torch.bfloat16)
    ids = torch.empty(rows, 2, dtype=torch.int32, device=DEV)
    w = torch.empty(rows, 2, device=DEV)
    moe.moe_router_topk(x[:, :64], ids, w)
    i7, w7 = torch.empty(7, 2, dtype=torch.int32, device=DEV), torch.empty(7, 2, device=DEV)
    moe.moe_router_topk(x[-7:, :64].contiguous(), i7, w7)
    torch.cuda.synchronize()
    assert torch.equal(ids[-7:], i7) and torch.equal(w[-7:], w7)
    assert (ids[:5] == torch.tensor([0, 1], device=DEV)).all()
    q = torch.empty(512, -(-rows // 128) * 128, dtype=torch.uint8, device=DEV)
    sf = torch.empty(512, -(-rows // 128), device=DEV)
    moe.moe_quant_act_t(x, q, sf)
    tail = x[rows // 128 * 128:].contiguous()
    q2, sf2 = torch.empty(512, 128, dtype=torch.uint8, device=DEV), torch.empty(512, 1, device=DEV)
    moe.moe_quant_act_t(tail, q2, sf2)
    torch.cuda.synchronize()
    assert torch.equal(q[:, -128:], q2) and torch.equal(sf[:, -1:], sf2) and not q[:, :-256].any()


def test_router_at_its_largest():
    """2^31 - 1 tokens of one expert: the row number ends just below 32 bits."""
    require_gpu()
    n = (1 << 31) - 1
    x = torch.zeros(n, 1, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((n, 1), 7, dtype=torch.int32, device=DEV)
    w = torch.zeros(n, 1, device=DEV)
    moe.moe_router_topk(x, ids, w, score="sigmoid", renormalize=False, scale=2.0)
    torch.cuda.synchronize()
    assert int(ids.max()) == 0 and int(ids.min()) == 0
    assert float(w.min()) == 1.0 and float(w.max()) == 1.0  # 2 * sigmoid(0)
    d = torch.full((n, 1), 9.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_router_topk_bwd(x, ids, w, d, score="sigmoid", renormalize=False, scale=2.0)
    torch.cuda.synchronize()
    assert float(d.min()) == 0.5 and float(d.max()) == 0.5  # 2 * 1 * 1/4
