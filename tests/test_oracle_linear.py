"""The oracle of the dense product with its epilogue: activations, slopes, a hand-written loop, gradients by differences."""

import numpy as np
import pytest
from scipy import special

import oracle

NAMES = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def test_activations_against_scipy():
    v = np.linspace(-12, 12, 2001)
    assert np.allclose(oracle.act("silu", v), v * special.expit(v), rtol=1e-13)
    assert np.allclose(oracle.act("gelu", v), v * special.ndtr(v), rtol=1e-12, atol=1e-300)
    u = np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
    assert np.allclose(oracle.act("gelu_tanh", v), 0.5 * v * (1 + np.tanh(u)), rtol=1e-9, atol=1e-14)
    assert np.array_equal(oracle.act("relu", v), np.where(v > 0, v, 0)) and np.array_equal(oracle.act("none", v), v)


@pytest.mark.parametrize("name", NAMES)
def test_slopes_against_differences(name):
    v = np.linspace(-7.03, 7.01, 501)
    d = (oracle.act(name, v + 1e-6) - oracle.act(name, v - 1e-6)) / 2e-6
    assert np.allclose(oracle.act_slope(name, v), d, atol=1e-8)


@pytest.mark.parametrize("gated", [False, True])
def test_product_by_loops(gated):
    g = np.random.default_rng(0)
    M, N, K = 3, 4, 5
    a, w, b = g.normal(size=(M, K)), g.normal(size=(N, K)), g.normal(size=N)
    c = g.normal(size=(M, N // 2 if gated else N))
    d, v, mag = oracle.linear(a, w, b, "silu", gated, c)
    for m in range(M):
        for n in range(N):
            s = sum(a[m, k] * w[n, k] for k in range(K)) + b[n]
            assert abs(v[m, n] - s) < 1e-12
            assert abs(mag[m, n] - sum(abs(a[m, k] * w[n, k]) for k in range(K)) - abs(b[n])) < 1e-12
        for n in range(c.shape[1]):
            silu = v[m, n] / (1 + np.exp(-v[m, n]))
            assert abs(d[m, n] - (silu * v[m, 2 + n] if gated else silu) - c[m, n]) < 1e-12


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_gradient_by_differences(name, gated):
    g = np.random.default_rng(1)
    pre = g.normal(size=(3, 8))
    dD = g.normal(size=(3, 4 if gated else 8))
    f = lambda p: ((oracle.act(name, p[:, :4]) * p[:, 4:] if gated else oracle.act(name, p)) * dD).sum()  # noqa: E731
    got = oracle.act_bwd(dD, pre, name, gated)
    for i in np.ndindex(pre.shape):
        p, q = pre.copy(), pre.copy()
        p[i] += 1e-6
        q[i] -= 1e-6
        assert abs((f(p) - f(q)) / 2e-6 - got[i]) < 1e-7
