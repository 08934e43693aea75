"""The dense product with bias, activation and residual, and its gradient, in float64.  TEST INFRASTRUCTURE ONLY.

Written from the definitions in include/moe.h (moe_gemm_bf16, moe_act_bwd).
"""

from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(v):
    t = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, t) / (1.0 + t)


def act(name: str, v: np.ndarray) -> np.ndarray:
    """Pinned by: values of scipy's expit and ndtr, and tanh's form of gelu_tanh."""
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v * _sigmoid(v)
    if name == "gelu":
        return v * 0.5 * _erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return v * _sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def act_slope(name: str, v: np.ndarray) -> np.ndarray:
    """Pinned by: central differences of act."""
    if name == "relu":
        return (v > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(v)
        return s + v * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * _erfc(-v / math.sqrt(2.0)) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = _sigmoid(c * (v + 0.044715 * v ** 3))
        return s + v * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * v * v)
    return np.ones_like(v)


def linear(a, w, bias=None, name="none", gated=False, residual=None):
    """(D, v, magnitude of v's products): a [M, K], w [N, K]."""
    v = a @ w.T
    mag = np.abs(a) @ np.abs(w).T
    if bias is not None:
        v, mag = v + bias, mag + np.abs(bias)
    h = v.shape[1] // 2
    d = act(name, v[:, :h]) * v[:, h:] if gated else act(name, v)
    return (d if residual is None else d + residual), v, mag


def act_bwd(dD, pre, name="none", gated=False):
    """dP [M, N] of dD and the pre-activation."""
    if not gated:
        return dD * act_slope(name, pre)
    h = dD.shape[1]
    gate, up = pre[:, :h], pre[:, h:]
    return np.concatenate((dD * up * act_slope(name, gate), dD * act(name, gate)), 1)
