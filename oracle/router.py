"""The router's choice, its weights and their gradient, in float64.  TEST INFRASTRUCTURE ONLY.

Written row by row from the definition (include/moe.h, moe_router_topk): scores, keys, group scores, the k
largest keys with ties to the lowest expert, weights as given or renormalised over the slots.
"""

from __future__ import annotations

import numpy as np


def router_scores(x: np.ndarray, score: str) -> np.ndarray:
    """Scores of one row; 0 for an expert that is not available (logit -inf or NaN).

    Pinned by: scipy's softmax and expit on finite rows.
    """
    x = np.asarray(x, dtype=np.float64)
    ok = ~(np.isnan(x) | (x == -np.inf))
    s = np.zeros_like(x)
    if not ok.any():
        return s
    if score == "sigmoid":
        t = np.exp(-np.abs(x[ok]))
        s[ok] = np.where(x[ok] >= 0, 1.0, t) / (1.0 + t)
    else:
        m = x[ok].max()
        e = np.where(x[ok] == m, 1.0, np.exp(np.where(x[ok] == m, 0.0, x[ok] - m)))
        s[ok] = e / e.sum()
    return s


def router_topk(logits, k, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True,
                scale=1.0):
    """(topk_ids int32 [T, k], topk_weights float64 [T, k]) of logits [T, E].

    Pinned by: a sort of every row (no groups), hand-worked groups, and ties.
    """
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    S = E // n_group
    ids = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        x = logits[t]
        s = router_scores(x, score)
        with np.errstate(invalid="ignore"):
            key = x.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
        none = np.isnan(x) | (x == -np.inf) | np.isnan(key) | (key == -np.inf)
        groups = []
        for g in range(n_group):
            mine = [e for e in range(g * S, (g + 1) * S) if not none[e]]
            v = key if group_top == 1 or bias is not None else s
            top = sorted((v[e] for e in mine), reverse=True)[:group_top]
            groups.append(sum(top) if top else -np.inf)
        kept = sorted(range(n_group), key=lambda g: (-groups[g], g))[:topk_group]
        cand = [e for g in sorted(kept) for e in range(g * S, (g + 1) * S) if not none[e]]
        order = sorted(cand, key=lambda e: (-key[e], e))[:k]
        ids[t, :len(order)] = order
    return ids, router_weights(logits, ids, score, renormalize, scale)


def router_weights(logits, ids, score="softmax", renormalize=True, scale=1.0) -> np.ndarray:
    """topk_weights float64 [T, k] of a choice; 0 for a slot without an available expert.

    Pinned by: router_scores, and the renormalised sum (scale).  The renormalised sigmoid is evaluated through
    log s = min(x, 0) - log(1 + exp(-|x|)), so it does not underflow.
    """
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    w = np.zeros(ids.shape, dtype=np.float64)
    for t in range(T):
        on = [(r, int(e)) for r, e in enumerate(ids[t]) if 0 <= e < E and logits[t, e] > -np.inf]
        if not on:
            continue
        x = np.array([logits[t, e] for _, e in on])
        if renormalize:
            logs = x if score == "softmax" else np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
            m = logs.max()
            q = np.exp(np.where(logs == m, 0.0, logs - m))
            q /= q.sum()
        else:
            q = router_scores(logits[t], score)[[e for _, e in on]]
        w[t, [r for r, _ in on]] = scale * q
    return w


def router_topk_bwd(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0) -> np.ndarray:
    """d logits float64 [T, E] of sum(dweights * router_weights(logits, ids)).

    Pinned by: central differences of router_weights.
    """
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    w = router_weights(logits, ids, score, renormalize, 1.0)
    d = np.zeros((T, E), dtype=np.float64)
    for t in range(T):
        on = [(r, int(e)) for r, e in enumerate(ids[t]) if 0 <= e < E and logits[t, e] > -np.inf]
        if not on:
            continue
        g = {r: scale * float(dweights[t, r]) for r, _ in on}
        mean = sum(g[r] * w[t, r] for r, _ in on)
        for r, e in on:
            c = w[t, r] * (g[r] - (mean if renormalize else 0.0))
            if score == "sigmoid":
                c *= router_scores(np.array([-logits[t, e]]), "sigmoid")[0]
            d[t, e] += c
        if score == "softmax" and not renormalize:
            d[t] -= router_scores(logits[t], "softmax") * mean
    return d
