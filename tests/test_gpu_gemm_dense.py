"""The dense FP8 product and the transposing quantiser on the GPU.

Bound of the product against the float64 sum: a block of 128 products is summed in fp32 by the matrix core (counted as
one truncation, 2^-23, per product: 2 * 128 units of 2^-24), its scales' product and its promotion round once each (2), the running sum
once per block, and the addend and a split's partial sums a few times more: (256 + 2 + K/128 + 8) * 2^-24 of
the sum of magnitudes.

bf16 output comes from the FP8 matrix instruction, which aligns each group of 8 products to the largest binade
2^e = 2^(ea + eb) among them and drops the bits below 2^(e - 13).  Each of the other 7 products loses less than
2^(e - 13), and the largest product of the group is at least 2^e, so the group loses less than 7 * 2^-13 of its largest
product, hence of its sum of magnitudes; this holds for every group, hence for the whole sum: 7 * 2^-13 = 14336 * 2^-24
of the sum of magnitudes more.  The rounding to bf16 adds half a step, 2^-8.

Where every partial sum is an integer multiple of one unit below 2^24 (and products differ by less than 2^13), the
result is exact.
"""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, require_gpu, u16

pytestmark = pytest.mark.gpu


def _ws(M, N, K, fill=0xA5):
    return torch.full((max(16, moe.moe_gemm_fp8_workspace_bytes(M, N, K)),), fill, dtype=torch.uint8, device=DEV)


def _operands(M, N, K, gran, seed):
    rng = np.random.default_rng(seed)
    tab = oracle.e4m3_decode_table()
    finite = np.nonzero(np.isfinite(tab))[0].astype(np.uint8)
    a, w = rng.choice(finite, (M, K)), rng.choice(finite, (N, K))
    # scales that are no powers of two, over several binades, one of them negative and one zero
    sa = np.exp(rng.uniform(-6, 3, (M, K // 128))).astype(np.float32)
    sw = np.exp(rng.uniform(-6, 3, (-(-N // gran), K // 128))).astype(np.float32)
    sa.flat[0] *= -1
    sw.flat[-1] = 0
    return a, sa, w, sw


def _t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _run(a, sa, w, sw, out, c=None, lda=0, ldw=0, ldd=0, d=None):
    M, K = a.shape
    N = w.shape[0]

    def wide(x, ld):
        if not ld:
            return _t(x)
        b = torch.full((x.shape[0], ld), 0x7F, dtype=torch.uint8, device=DEV)  # NaN codes around the rows
        b[:, :x.shape[1]] = _t(x)
        return b[:, :x.shape[1]]

    D = torch.full((M, ldd or N), 77.0, dtype=out, device=DEV) if d is None else d
    moe.moe_gemm_fp8(wide(a, lda), _t(sa), wide(w, ldw), _t(sw), D[:, :N], C=None if c is None else c,
                     workspace=_ws(M, N, K))
    torch.cuda.synchronize()
    assert (D[:, N:] == 77.0).all(), "written past column N"
    return D[:, :N]


def _check(d, a, sa, w, sw, gran, c=None):
    ref, mag = oracle.dense_gemm_fp8(a, sa, w, sw, gran, c)
    K = a.shape[1]
    got = d.float().cpu().numpy().astype(np.float64)
    bf = d.dtype == torch.bfloat16
    half = 2.0 ** -8 if bf else 0.0
    tol = (266 + K // 128 + (7 * 2 ** 11 if bf else 0)) * 2.0 ** -24 * mag
    bad = np.abs(got - ref) > tol + half * (np.abs(ref) + tol) + 1e-38
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, first {np.argwhere(bad)[0]}"


SIZES = [(1, 1, 128), (1, 64, 256), (1, 4096, 1024), (2, 130, 384), (7, 33, 128), (16, 16, 2048), (17, 257, 640),
         (31, 1000, 512), (33, 128, 128), (64, 320, 1152), (65, 127, 256), (100, 96, 7168), (129, 129, 896),
         (200, 640, 384), (255, 513, 128), (257, 250, 256), (300, 1100, 640), (512, 384, 512), (777, 259, 384), (40, 5000, 384), (5, 4200, 1280),
         (20, 4500, 640), (66, 300, 4096), (130, 64, 32768), (1100, 3000, 384), (1030, 4100, 256), (2100, 4500, 640), (70, 3000, 1280), (259, 1300, 640), (577, 800, 896),
         (131, 2200, 7168), (1000, 130, 512), (4000, 64, 7168), (4000, 60, 512)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("gran", [128, 1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_against_oracle(M, N, K, gran, out):
    require_gpu()
    a, sa, w, sw = _operands(M, N, K, gran, M * 7 + N + K)
    _check(_run(a, sa, w, sw, out), a, sa, w, sw, gran)


@pytest.mark.parametrize("M,N,K", [(1, 70, 256), (19, 130, 512), (140, 300, 384), (300, 513, 256)])
@pytest.mark.parametrize("gran", [128, 1])
def test_addend_and_strides(M, N, K, gran):
    require_gpu()
    a, sa, w, sw = _operands(M, N, K, gran, M + N)
    c = np.random.default_rng(1).standard_normal((M, N)).astype(np.float32) * 50
    cw = torch.full((M, N + 5), float("nan"), device=DEV)
    cw[:, :N] = _t(c)
    for ldd in (0, N + 3, N + 4):
        _check(_run(a, sa, w, sw, torch.float32, cw[:, :N], K + 16, K + 48, ldd), a, sa, w, sw, gran, c)
        _check(_run(a, sa, w, sw, torch.bfloat16, None, K + 32, K + 16, ldd), a, sa, w, sw, gran)
    inplace = _t(c)
    first = _run(a, sa, w, sw, torch.float32, _t(c))
    assert torch.equal(_run(a, sa, w, sw, torch.float32, inplace, d=inplace), first)  # C is D


@pytest.mark.parametrize("M,N,K", [(1, 300, 7168), (24, 200, 4096), (130, 500, 1024), (520, 768, 256)])
@pytest.mark.parametrize("gran", [128, 1])
def test_exact_on_integers(M, N, K, gran):
    """Codes 0, +-1, +-2 and scales 1, 2 or 3: every sum is a whole number below 2^24."""
    require_gpu()
    rng = np.random.default_rng(N)
    codes = np.array([0x00, 0x38, 0xB8, 0x40, 0xC0], np.uint8)
    a, w = rng.choice(codes, (M, K)), rng.choice(codes, (N, K))
    sa = rng.integers(1, 4, (M, K // 128)).astype(np.float32)
    sw = rng.integers(1, 4, (-(-N // gran), K // 128)).astype(np.float32)
    ref, mag = oracle.dense_gemm_fp8(a, sa, w, sw, gran)
    assert mag.max() < 2 ** 24
    assert np.array_equal(_run(a, sa, w, sw, torch.float32).cpu().numpy().astype(np.float64), ref)


def test_powers_of_two_match_the_grouped_product():
    """One expert, power-of-two scales: both products round the same exact values (within the two bounds)."""
    require_gpu()
    M, N, K = 150, 256, 512
    x = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    wt = (torch.randn(1, N, K, device=DEV) * 0.05).to(torch.bfloat16)
    q, sf = torch.empty(M, K, dtype=torch.uint8, device=DEV), torch.empty(M, K // 128, device=DEV)
    wq, ws = torch.empty(1, N, K, dtype=torch.uint8, device=DEV), torch.empty(1, N // 128, K // 128, device=DEV)
    moe.moe_quant_act(x, q, sf)
    moe.moe_quant_weight_fp8(wt, wq, ws)
    D = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_gemm_fp8(q, sf, wq[0], ws[0], D, workspace=_ws(M, N, K))
    G = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    cnt = torch.tensor([M], dtype=torch.int32, device=DEV)
    seg = torch.tensor([0, M], dtype=torch.int32, device=DEV)
    moe.moe_grouped_gemm_fp8(moe.LAYOUT_CONTIGUOUS, q, sf, wq, ws, G, cnt, seg, 1, M, N, K)
    torch.cuda.synchronize()
    a, w = q.cpu().numpy(), wq[0].cpu().numpy()
    for d in (D, G):
        _check(d, a, sf.cpu().numpy(), w, ws[0].cpu().numpy(), 128)


@pytest.mark.parametrize("M", [10, 40, 140, 600])
def test_special_values_bf16(M):
    """The same in bf16 output, on every kernel's path."""
    require_gpu()
    N, K = 1100, 512
    a, sa, w, sw = _operands(M, N, K, 128, M)
    sa, sw = np.abs(sa) + 0.1, np.abs(sw) + 0.1
    clean = _run(a, sa, w, sw, torch.bfloat16)
    a2, w2 = a.copy(), w.copy()
    a2[M - 3, 129] = 0xFF
    w2[1050, 511] = 0x7F
    d = _run(a2, sa, w2, sw, torch.bfloat16)
    rows, cols = torch.arange(M) != M - 3, torch.arange(N) != 1050
    assert torch.isnan(d[M - 3]).all() and torch.isnan(d[:, 1050]).all()
    assert torch.equal(d[rows][:, cols], clean[rows][:, cols])


def test_special_values():
    """A NaN code reaches its row (or column) only; an infinite scale likewise; rows stay apart."""
    require_gpu()
    M, N, K = 40, 150, 256
    a, sa, w, sw = _operands(M, N, K, 1, 3)
    sa, sw = np.abs(sa), np.abs(sw) + 0.1
    clean = _run(a, sa, w, sw, torch.float32)
    a2 = a.copy()
    a2[5, 200] = 0x7F
    d = _run(a2, sa, w, sw, torch.float32)
    assert torch.isnan(d[5]).all()
    keep = torch.arange(M) != 5
    assert torch.equal(d[keep], clean[keep])
    w2 = w.copy()
    w2[149, 0] = 0xFF
    d = _run(a, sa, w2, sw, torch.float32)
    assert torch.isnan(d[:, 149]).all() and torch.equal(d[:, :149], clean[:, :149])
    s2 = sa.copy()
    s2[7, 1] = np.inf
    d = _run(a, s2, w, sw, torch.float32)
    assert not torch.isfinite(d[7]).any()
    keep = torch.arange(M) != 7
    assert torch.equal(d[keep], clean[keep])


def test_deterministic_and_workspace_is_not_read():
    require_gpu()
    for M, N, K in ((1, 512, 7168), (30, 256, 4096), (131, 1024, 2048), (260, 300, 1024)):
        a, sa, w, sw = (_t(v) for v in _operands(M, N, K, 128, M))
        outs = []
        for fill in (0x00, 0xFF, 0x7F):
            D = torch.empty(M, N, dtype=torch.float32, device=DEV)
            moe.moe_gemm_fp8(a, sa, w, sw, D, workspace=_ws(M, N, K, fill))
            outs.append(D)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_empty_and_refusals():
    require_gpu()
    u = torch.zeros(4, 256, dtype=torch.uint8, device=DEV)
    s = torch.ones(4, 2, device=DEV)
    d = torch.ones(4, 4, device=DEV)
    moe.moe_gemm_fp8(u[:0], s[:0], u, s, d[:0])
    for args, kw in (((u, s, u, s[:, :1].contiguous(), d), {}), ((u, s, u[:3], s, d), {}), ((u, s[:3], u, s, d), {}),
                     ((u, s, u, s, d.half()), {}), ((u.t(), s, u, s, d), {}), ((u, s, u, s, d), dict(C=d[:3])),
                     ((u, s, u, s, d), dict(C=d.to(torch.bfloat16)))):
        with pytest.raises(ValueError):
            moe.moe_gemm_fp8(*args, workspace=_ws(4, 4, 256), **kw)
    with pytest.raises(moe.MoeError):
        moe.moe_gemm_fp8(u, s, u, s, d.to(torch.bfloat16), C=d, workspace=_ws(4, 4, 256))
    with pytest.raises(moe.MoeError):
        moe.moe_gemm_fp8(u[:, 8:136], s[:, :1].contiguous(), u[:, :128], s[:, :1].contiguous(), d, workspace=_ws(4, 4, 128))


# ------------------------------------------------------------------ transposing quantiser --
@pytest.mark.parametrize("M,K", [(1, 8), (5, 64), (127, 72), (128, 128), (129, 1536), (300, 40), (333, 200), (1000, 264)])
def test_quant_act_t(M, K):
    require_gpu()
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-20, 20, (M, K), generator=g).float())
    x[:, 3] = 0
    x[0, 5] = -0.0
    x = x.to(torch.bfloat16)
    mb = -(-M // 128)
    for ld in (K, K + 24):
        xs = torch.full((M, ld), float("nan"), dtype=torch.bfloat16, device=DEV)
        xs[:, :K] = x.to(DEV)
        q = torch.full((K, 128 * mb), 0x55, dtype=torch.uint8, device=DEV)
        sf = torch.full((K, mb), -1.0, device=DEV)
        moe.moe_quant_act_t(xs[:, :K], q, sf)
        torch.cuda.synchronize()
        rq, rs = oracle.quant_act_t(u16(x))
        assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(sf.cpu().numpy(), rs)


def test_quant_act_t_is_quant_act_of_the_transpose():
    """Every bf16 pattern: subnormals, zeros, infinities and quiet NaN in every block."""
    require_gpu()
    g = torch.Generator().manual_seed(1)
    bits = torch.randint(0, 65536, (1280, 256), generator=g, dtype=torch.int32)
    nan = ((bits & 0x7F80) == 0x7F80) & ((bits & 0x7F) != 0)
    bits = torch.where(nan, bits | 0x40, bits)
    bits[:128] &= 0x807F  # subnormals alone
    bits[128:256] &= 0x8000  # zeros of both signs
    bits[256:768] = torch.where((bits[256:768] & 0x7F80) == 0x7F80, 0x3F80, bits[256:768])  # finite alone
    x = bits.to(torch.int16).view(torch.bfloat16).to(DEV)
    q, sf = torch.empty(256, 1280, dtype=torch.uint8, device=DEV), torch.empty(256, 10, device=DEV)
    moe.moe_quant_act_t(x, q, sf)
    q2, sf2 = torch.empty_like(q), torch.empty_like(sf)
    moe.moe_quant_act(x.t().contiguous(), q2, sf2)
    torch.cuda.synchronize()
    assert torch.equal(sf.view(torch.int32), sf2.view(torch.int32)) and torch.equal(q, q2)


def test_quant_act_t_refusals():
    require_gpu()
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device=DEV)
    q, sf = torch.empty(16, 128, dtype=torch.uint8, device=DEV), torch.empty(16, 1, device=DEV)
    moe.moe_quant_act_t(x[:0], q[:, :0].contiguous(), sf[:, :0].contiguous())
    with pytest.raises(ValueError):
        moe.moe_quant_act_t(x, q[:15].contiguous(), sf)
    with pytest.raises(ValueError):
        moe.moe_quant_act_t(x.float(), q, sf)
    with pytest.raises(moe.MoeError):
        moe.moe_quant_act_t(torch.zeros(4, 20, dtype=torch.bfloat16, device=DEV)[:, 4:], q, sf)  # rows not 16-byte aligned
    with pytest.raises(moe.MoeError):
        moe.moe_quant_act_t(torch.zeros(4, 12, dtype=torch.bfloat16, device=DEV),
                            torch.empty(12, 128, dtype=torch.uint8, device=DEV), torch.empty(12, 1, device=DEV))
