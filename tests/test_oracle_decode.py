"""The oracle of the few-token expert layer against a hand-written loop and the combine's own oracle (CPU)."""

import numpy as np

import oracle


def test_experts_by_loops():
    g = np.random.default_rng(0)
    T, k, E, H, I = 3, 2, 4, 6, 5
    x, p = g.normal(size=(T, H)), g.random((T, k))
    ids = np.array([[0, 3], [2, 2], [-1, 4]])  # an expert twice, a skipped slot, one out of range
    w13, w2, c = g.normal(size=(E, 2 * I, H)), g.normal(size=(E, H, I)), g.normal(size=(T, H))
    z, bound = oracle.experts_decode(x, ids, p, w13, w2, c)
    ref = c.copy()
    for t in range(T):
        for r in range(k):
            e = ids[t, r]
            if e < 0 or e >= E:
                continue
            for n in range(H):
                s = 0.0
                for j in range(I):
                    gate = sum(w13[e, j, q] * x[t, q] for q in range(H))
                    up = sum(w13[e, I + j, q] * x[t, q] for q in range(H))
                    s += w2[e, n, j] * gate / (1 + np.exp(-gate)) * up
                ref[t, n] += p[t, r] * s
    assert np.allclose(z, ref, rtol=1e-12) and (bound == 0).all()
    assert np.array_equal(z[2], c[2])


def test_experts_as_a_combine():
    g = np.random.default_rng(1)
    T, k, E, H, I = 5, 3, 6, 8, 4
    x, p = g.normal(size=(T, H)), g.random((T, k))
    ids = np.argsort(g.random((T, E)), 1)[:, :k]
    w13, w2 = g.normal(size=(E, 2 * I, H)), g.normal(size=(E, H, I))
    rows = np.stack([w2[e] @ oracle.swiglu((w13[e] @ x[t])[None])[0] for t in range(T) for e in ids[t]])
    z, _ = oracle.experts_decode(x, ids, p, w13, w2)
    assert np.allclose(z, oracle.combine(rows, np.arange(T * k).reshape(T, k), p), rtol=1e-12)


def test_bound_covers_a_perturbation():
    """Errors of the stated sizes, put in on purpose, stay within the bound."""
    g = np.random.default_rng(2)
    T, k, E, H, I = 4, 2, 3, 16, 8
    x, p = g.normal(size=(T, H)), g.random((T, k))
    ids = g.integers(0, E, (T, k))
    w13, w2 = g.normal(size=(E, 2 * I, H)), g.normal(size=(E, H, I))
    eps = 2.0 ** -8
    z, bound = oracle.experts_decode(x, ids, p, w13, w2, rounding=eps)
    got = np.zeros_like(z)
    for t in range(T):
        for r in range(k):
            e = ids[t, r]
            h = oracle.swiglu((w13[e] @ x[t])[None])[0]
            got[t] += p[t, r] * (w2[e] @ (h * (1 + eps * g.choice([-1, 1], I))))
    assert (np.abs(got - z) <= bound * (1 + 1e-9)).all()
