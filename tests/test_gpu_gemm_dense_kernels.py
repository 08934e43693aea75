"""Every kernel of the dense FP8 product over a long K, bit by bit.

Codes 0, +-1 and +-2 and scales 1/2, 1 and 2: every product and every partial sum is a multiple of 1/4 whose magnitude
stays below 16 K (at most 120832 here, so below 2^24 quarters), and products differ by a factor of 4 at most, far
within the 2^13 that the FP8 matrix instruction keeps.  So each sum is exact in fp32 in any order, fp32 output equals the float64 sum
and bf16 output that sum rounded once: a single product, block or scale missed, doubled or taken from the wrong slot shows.
"""

import pytest
import torch

import dense_shapes
import int4_weights_amd as moe
from gpu_helpers import DEV, require_gpu

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, gran, seed, offset=0):
    """offset: the scales begin that many floats past a 16-byte boundary."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device=DEV)
    vals = torch.tensor([0.5, 1.0, 2.0], device=DEV)

    def scales(rows):
        s = torch.empty(rows * (K // 128) + offset, device=DEV)[offset:].view(rows, K // 128)
        s.copy_(vals[torch.randint(0, 3, s.shape, generator=g, device=DEV)])
        return s

    a = codes[torch.randint(0, 5, (M, K), generator=g, device=DEV)]
    w = codes[torch.randint(0, 5, (N, K), generator=g, device=DEV)]
    return a, scales(M), w, scales(-(-N // gran))


def _exact(a, sa, w, sw, gran):
    def values(c, s, n):
        return c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(n, 0)[:c.shape[0]].repeat_interleave(128, 1)

    return values(a, sa, 1) @ values(w, sw, gran).t()


def _ws(M, N, K, fill):
    return torch.full((max(16, moe.moe_gemm_fp8_workspace_bytes(M, N, K)),), fill, dtype=torch.uint8, device=DEV)


def _check(M, N, K, f32, gran, offset=0):
    a, sa, w, sw = _inputs(M, N, K, gran, M + N + K + gran, offset)
    ref = _exact(a, sa, w, sw, gran)
    want = ref.float().to(torch.float32 if f32 else torch.bfloat16)
    for fill in (0x00, 0xFF, 0x7F):  # whatever the workspace holds
        D = torch.full((M, N), 77.0, dtype=want.dtype, device=DEV)
        moe.moe_gemm_fp8(a, sa, w, sw, D, workspace=_ws(M, N, K, fill))
        torch.cuda.synchronize()
        assert torch.equal(D, want), f"{int((D != want).sum())} of {D.numel()} differ"
    if f32:
        C = torch.randint(-1000, 1000, (M, N), device=DEV).float()
        D = C.clone()
        moe.moe_gemm_fp8(a, sa, w, sw, D, C=D, workspace=_ws(M, N, K, 0xFF))
        torch.cuda.synchronize()
        assert torch.equal(D, want + C)


@pytest.mark.parametrize("M,N,K,f32,kind,splits", dense_shapes.ALL)
@pytest.mark.parametrize("gran", [128, 1])
def test_exact(M, N, K, f32, kind, splits, gran):
    require_gpu()
    _check(M, N, K, f32, gran)


@pytest.mark.parametrize("M,N,K,f32,kind,splits", [s for s in dense_shapes.ALL if s[2] in (2048, 7168)])
def test_scales_that_cannot_be_copied_as_vectors(M, N, K, f32, kind, splits):
    require_gpu()
    _check(M, N, K, f32, 1, offset=1)


ONE_EACH = list({(s[3], s[4], s[5] > 1): s for s in dense_shapes.ALL if s[2] >= 2048}.values())


@pytest.mark.parametrize("M,N,K,f32,kind,splits", ONE_EACH)
def test_nan_and_infinite_scales_stay_in_their_row_and_column(M, N, K, f32, kind, splits):
    require_gpu()
    a, sa, w, sw = _inputs(M, N, K, 1, M + N)
    out = torch.float32 if f32 else torch.bfloat16

    def run():
        D = torch.empty(M, N, dtype=out, device=DEV)
        moe.moe_gemm_fp8(a, sa, w, sw, D, workspace=_ws(M, N, K, 0xFF))
        return D

    clean = run()
    rows, cols = [0, M // 2, M - 1], [1, N // 2, N - 1]
    a[rows[0], K - 1] = 0x7F  # NaN codes, of either sign, in the first and last block
    a[rows[1], 3] = 0xFF
    w[cols[0], K - 130] = 0xFF
    w[cols[1], 0] = 0x7F
    sa[rows[2], K // 128 - 1] = float("inf")
    sw[cols[2], 5] = float("nan")
    d = run()
    torch.cuda.synchronize()
    keep_r = torch.ones(M, dtype=torch.bool, device=DEV)
    keep_c = torch.ones(N, dtype=torch.bool, device=DEV)
    keep_r[rows], keep_c[cols] = False, False
    assert not torch.isfinite(d[~keep_r]).any() and torch.isnan(d[:, ~keep_c]).all()
    assert torch.equal(d[keep_r][:, keep_c], clean[keep_r][:, keep_c])


@pytest.mark.parametrize("M", [9, 131, 300, 1100])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_that_cancel(M, out):
    """Pairs of +-448 * 448 beside products of 1/4 to 1, which the sums consist of.  fp32 output counts every product: it is
    within (2 * 128 + 2 + K / 128 + 8) units of 2^-24 of the sum of magnitudes, as for any data.  bf16 output loses at
    most 7 * 2^-13 of it more (each of a group's 7 smaller products less than 2^-13 of the largest's binade), and half a step.
    """
    require_gpu()
    N, K = 160, 1024
    g = torch.Generator(device=DEV).manual_seed(M)
    small = torch.tensor([0x30, 0xB0, 0x38, 0xB8], dtype=torch.uint8, device=DEV)  # +-0.5, +-1
    a = small[torch.randint(0, 4, (M, K), generator=g, device=DEV)]
    w = small[torch.randint(0, 4, (N, K), generator=g, device=DEV)]
    a[:, 0::4], a[:, 1::4] = 0x7E, 0x7E
    w[:, 0::4], w[:, 1::4] = 0x7E, 0xFE
    sa, sw = torch.ones(M, K // 128, device=DEV), torch.ones(2, K // 128, device=DEV)
    x, y = a.view(torch.float8_e4m3fn).double(), w.view(torch.float8_e4m3fn).double()
    ref, mag = x @ y.t(), x.abs() @ y.abs().t()
    D = torch.empty(M, N, dtype=out, device=DEV)
    moe.moe_gemm_fp8(a, sa, w, sw, D, workspace=_ws(M, N, K, 0xFF))
    torch.cuda.synchronize()
    tol = ((7 * 2 ** 11 if out is torch.bfloat16 else 0) + 266 + K // 128) * 2.0 ** -24 * mag
    half = 2.0 ** -8 if out is torch.bfloat16 else 0.0
    assert ((D.double() - ref).abs() <= tol + half * (ref.abs() + tol)).all()


def test_two_streams_with_shares_of_k_and_row_tables():
    """A product whose K is shared and a combine gradient of more than 4096 routes on each of two streams at once, each
    with a workspace of its own."""
    require_gpu()
    M, N, K, T, k, n = 131, 256, 7168, 1300, 4, 256
    assert moe.moe_gemm_fp8_workspace_bytes(M, N, K) > 0
    assert moe.moe_unpermute_combine_bwd_workspace_bytes(T, k, T * k) > 0
    sets = []
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        a, sa, w, sw = _inputs(M, N, K, 128, seed)
        dz = torch.randn(T, n, generator=g).to(torch.bfloat16).to(DEV)
        y = torch.randn(T * k, n, generator=g).to(torch.bfloat16).to(DEV)
        oi = torch.randperm(T * k, generator=g).view(T, k).to(torch.int32).to(DEV)
        tw = torch.rand(T, k, generator=g).to(DEV)
        D, dY, dw = torch.empty(M, N, device=DEV), torch.empty_like(y), torch.empty(T, k, device=DEV)
        cws = torch.empty(moe.moe_unpermute_combine_bwd_workspace_bytes(T, k, T * k), dtype=torch.uint8, device=DEV)
        sets.append((torch.cuda.Stream(), (a, sa, w, sw, D), _ws(M, N, K, 0xFF), (dz, y, oi, tw, dY, dw), cws))

    def outputs():
        return [t for _, p, _, c, _ in sets for t in (p[4], c[4], c[5])]

    def issue(s, p, ws, c, cws):
        moe.moe_gemm_fp8(*p, workspace=ws, stream=s)
        moe.moe_unpermute_combine_bwd(*c, workspace=cws, stream=s)

    for one in sets:  # one after the other
        torch.cuda.synchronize()
        issue(*one)
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs()]
    for (a, sa, w, sw, D), ref in zip([s[1] for s in sets], (want[0], want[3])):
        assert torch.equal(ref, _exact(a, sa, w, sw, 128).float())
    for _ in range(10):
        for t in outputs():
            t.fill_(5.0)
        torch.cuda.synchronize()
        for _ in range(3):
            for one in sets:
                issue(*one)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outputs(), want))
