"""Pins of the router's, the combine gradient's, the dense product's and the transposing quantiser's oracle."""

import numpy as np
import pytest
import scipy.special

import oracle


def test_scores_match_scipy():
    x = np.random.default_rng(0).standard_normal((20, 33)) * 4
    for row in x:
        assert np.allclose(oracle.router_scores(row, "softmax"), scipy.special.softmax(row), rtol=1e-14)
        assert np.allclose(oracle.router_scores(row, "sigmoid"), scipy.special.expit(row), rtol=1e-14)


def test_choice_without_groups_is_a_sort():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((30, 17))
    ids, w = oracle.router_topk(x, 5)
    assert np.array_equal(ids, np.argsort(-x, axis=1, kind="stable")[:, :5])
    assert np.allclose(w.sum(1), 1.0)
    b = rng.standard_normal(17)
    ids, w = oracle.router_topk(x, 5, score="sigmoid", bias=b, renormalize=False, scale=2.0)
    s = scipy.special.expit(x)
    assert np.array_equal(ids, np.argsort(-(s + b), axis=1, kind="stable")[:, :5])
    assert np.allclose(w, 2.0 * np.take_along_axis(s, ids, 1))


def test_groups_worked_by_hand():
    # 3 groups of 3: largest logits 5, 4, 3; sums of the two largest sigmoids order them 2, 1, 0
    x = np.array([[5.0, -9.0, -9.0, 4.0, 1.0, -9.0, 3.0, 3.0, 2.0]])
    ids, _ = oracle.router_topk(x, 3, score="sigmoid", n_group=3, topk_group=2, group_top=1)
    assert ids.tolist() == [[0, 3, 4]]
    ids, _ = oracle.router_topk(x, 3, score="sigmoid", n_group=3, topk_group=2, group_top=2)
    assert ids.tolist() == [[3, 6, 7]]


def test_ties_and_unavailable_experts():
    x = np.array([[1.0, 2.0, 2.0, 1.0], [-np.inf, np.nan, 0.0, -np.inf], [-np.inf] * 4])
    ids, w = oracle.router_topk(x, 3)
    assert ids.tolist() == [[1, 2, 0], [2, -1, -1], [-1, -1, -1]]
    assert w[1].tolist() == [1.0, 0.0, 0.0] and w[2].tolist() == [0.0, 0.0, 0.0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 9)) * 2
    ids = np.argsort(-x, axis=1)[:, :4].astype(np.int32)
    ids[1, 2] = -1
    ids[2, 3] = ids[2, 0]  # one expert in two slots
    g = rng.standard_normal(ids.shape)
    d = oracle.router_topk_bwd(x, ids, g, score, renorm, 2.5)
    h = 1e-5
    for t in range(4):
        for e in range(9):
            xp, xm = x.copy(), x.copy()
            xp[t, e] += h
            xm[t, e] -= h
            num = (g * (oracle.router_weights(xp, ids, score, renorm, 2.5)
                        - oracle.router_weights(xm, ids, score, renorm, 2.5))).sum() / (2 * h)
            assert abs(num - d[t, e]) < 1e-8


def test_combine_gradient_is_the_adjoint():
    rng = np.random.default_rng(3)
    y, v = rng.standard_normal((12, 8)), rng.standard_normal((12, 8))
    oi = rng.integers(-1, 14, (5, 3)).astype(np.int32)  # repeated rows, skipped and out-of-range slots
    w, u = rng.standard_normal((5, 3)), rng.standard_normal((5, 3))
    dz = rng.standard_normal((5, 8))
    dy, named, dw = oracle.combine_bwd(dz, y, oi, w)
    assert np.isclose((dz * oracle.combine(v, oi, w)).sum(), (dy * v).sum())
    assert np.isclose((dz * oracle.combine(y, oi, u)).sum(), (dw * u).sum())
    assert set(np.nonzero(named)[0]) == {int(p) for p in oi.reshape(-1) if 0 <= p < 12}


def test_dense_product_against_loops_and_the_grouped_oracle():
    rng = np.random.default_rng(4)
    a = rng.integers(0, 127, (3, 256)).astype(np.uint8)
    w = rng.integers(0, 127, (130, 256)).astype(np.uint8)
    tab = oracle.e4m3_decode_table()
    for gran in (1, 128):
        sa = rng.uniform(0.5, 2, (3, 2)).astype(np.float32)
        sw = rng.uniform(0.5, 2, (130 if gran == 1 else 2, 2)).astype(np.float32)
        d, mag = oracle.dense_gemm_fp8(a, sa, w, sw, gran)
        for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
            ref = sum(float(sa[m, k // 128]) * float(sw[n // gran, k // 128]) * tab[a[m, k]] * tab[w[n, k]]
                      for k in range(256))
            assert np.isclose(d[m, n], ref, rtol=1e-13) and mag[m, n] >= abs(ref) * (1 - 1e-12)
    sa = np.exp2(rng.integers(-3, 3, (3, 2))).astype(np.float32)
    sw = np.exp2(rng.integers(-3, 3, (1, 2))).astype(np.float32)
    d, _ = oracle.dense_gemm_fp8(a, sa, w[:128], sw, 128)
    g = oracle.grouped_gemm_fp8(a, sa, w[None, :128], sw[None], np.array([3]), np.array([0, 3]))
    assert np.allclose(d, g[:3], rtol=1e-13)


def test_transposing_quantiser_pads_with_zeros():
    import torch
    x = torch.randn(130, 8).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    q, s = oracle.quant_act_t(x)
    assert q.shape == (8, 256) and s.shape == (8, 2)
    assert (q[:, 130:] == 0).all()
    q1, s1 = oracle.quant_act(np.ascontiguousarray(x[:128].T))
    assert np.array_equal(q[:, :128], q1) and np.array_equal(s[:, :1], s1)
