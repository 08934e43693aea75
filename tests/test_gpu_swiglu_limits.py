"""SwiGLU's far gates: every bf16 gate against the oracle, the largest ones (whose product with log2(e) overflows fp32) too."""

import numpy as np
import pytest
import torch

import int4_weights_amd as moe
import oracle
from gpu_helpers import DEV, bf16_from_u16, check_swiglu_quant, require_gpu

pytestmark = pytest.mark.gpu


def test_every_finite_gate():
    """One row per 128 gates of like size; the up value takes the row's results to about 1 (where fp32 holds silu at all)."""
    require_gpu()
    mag = np.arange(0x7F80, dtype=np.uint16)  # 0 to the largest finite number
    bits = np.stack((mag, mag | 0x8000)).reshape(2, -1, 128).reshape(-1, 128)
    rows = bits.shape[0]
    gate = oracle.bf16_bits_to_f64(bits)
    largest = np.abs(oracle.silu(gate)).max(1, keepdims=True)
    e = np.where(largest < 2.0 ** -126, 0.0, np.clip(-np.floor(np.log2(np.maximum(largest, 1e-300))), -126, 127))
    up = oracle.f32_to_bf16_bits(np.broadcast_to(np.exp2(e), bits.shape).astype(np.float32))
    gu = np.concatenate((bits, up), 1)
    q = torch.full((rows, 128), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full((rows, 1), -3.0, dtype=torch.float32, device=DEV)
    moe.moe_swiglu_quant(moe.LAYOUT_CONTIGUOUS, bf16_from_u16(gu), rows, torch.tensor([rows], dtype=torch.int32, device=DEV),
                         torch.tensor([0, rows], dtype=torch.int32, device=DEV), 1, q, sf)
    # (of all bf16 gates 4.2% lie within 1e-6 of a rounding midpoint, most of them on it)
    check_swiglu_quant(gu, q.cpu().numpy(), sf.cpu().numpy(), np.ones(rows, bool), 0xA5, -3.0, rare=0.05)
    top = gate[:, 0] > 2.0 ** 126  # and plainly: silu(g) = g there
    value = oracle.dequant_act(q.cpu().numpy(), sf.cpu().numpy())
    want = (gate * np.exp2(e))[top]
    assert top.any() and (np.abs(value[top] - want) <= 2.0 ** -4 * np.abs(want)).all()
