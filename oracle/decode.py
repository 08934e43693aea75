"""The expert layer of a few tokens, in float64.  TEST INFRASTRUCTURE ONLY.

Written from the definition in include/moe.h (moe_experts_decode), on values, not codes.
"""

from __future__ import annotations

import numpy as np

from .activation import silu


def experts_decode(x, ids, p, w13, w2, residual=None, rounding=0.0, accumulation=0.0, w_extra=0.0):
    """(Z, bound): x [T, H], ids and p [T, k], w13 [E, 2I, H], w2 [E, H, I] in float64.

    bound: how far a computation may be off whose h carries a relative error of `rounding` and whose sums carry
    `accumulation` times their products' magnitudes (weights counted w_extra larger where they are added up
    around an offset), by the triangle inequality.

    Pinned by: a loop over routes written out for one token, and the combine of separately computed experts.
    """
    T, H = x.shape
    I = w2.shape[2]
    z = np.zeros((T, H)) if residual is None else np.array(residual, dtype=np.float64)
    bound = np.zeros((T, H))
    for t in range(T):
        for r in range(ids.shape[1]):
            e = int(ids[t, r])
            if not 0 <= e < w13.shape[0]:
                continue
            gu = w13[e] @ x[t]
            mag = (np.abs(w13[e]) + w_extra) @ np.abs(x[t])
            h = silu(gu[:I]) * gu[I:]
            y = w2[e] @ h
            z[t] += p[t, r] * y
            # |silu'| <= 1.1
            dh = rounding * np.abs(h) + accumulation * (1.1 * mag[:I] * np.abs(gu[I:]) + np.abs(silu(gu[:I])) * mag[I:])
            bound[t] += abs(p[t, r]) * (np.abs(w2[e]) @ dh + accumulation * ((np.abs(w2[e]) + w_extra) @ np.abs(h)))
    return z, bound
