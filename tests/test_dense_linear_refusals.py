"""DenseFP8Linear's own checks of arguments (CPU: they come before any kernel)."""

import pytest
import torch

from int4_weights_amd.layer import DenseFP8Linear


@pytest.mark.parametrize("ty,tx", [(100, 120), (120, 100), (0, 5), (5, 0), (129, 128)])
@pytest.mark.parametrize("accumulate", [True, False])
def test_grad_weight_of_unequal_batches(ty, tx, accumulate):
    """dy and x of the same step have the same tokens; up to a block of 128 the codes' shapes do not tell."""
    m = DenseFP8Linear(torch.zeros(128, 256, dtype=torch.uint8), torch.ones(1, 2), 200)
    dw = torch.full((128, 256), 2.0)
    with pytest.raises(ValueError, match="tokens"):
        m.grad_weight(torch.zeros(ty, 128, dtype=torch.bfloat16), torch.zeros(tx, 256, dtype=torch.bfloat16), dw,
                      accumulate=accumulate)
    assert (dw == 2).all()
