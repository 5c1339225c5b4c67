"""Refusals of the Python binding of a training step's operators (CPU)."""
import pytest
import torch

import sparse_moe_layer_gate_amd as moe

CFG = moe.make_config(64, 16, 1, 1, 2, 64)


@pytest.mark.parametrize("mask", [[1, 1, 0, 1], (True,) * 4, 1, torch.ones(4, dtype=torch.bool), torch.ones(4)])
def test_token_mask_that_is_no_device_tensor(mask):
    with pytest.raises(TypeError, match="token_mask"):
        moe.moe_balance_loss(CFG, 4, None, None, 4, 0.1, None, None, None, None, token_mask=mask)
    with pytest.raises(TypeError, match="token_mask"):
        moe.moe_route_backward(CFG, 4, None, None, None, None, token_mask=mask)
