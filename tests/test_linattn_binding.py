"""The binding's checks of the layer norm's bias (CPU: refused before any pointer is taken)."""
import pytest
import torch

import gated_delta_rule_58_amd as kda


def test_layernorm_backward_checks_the_bias():
    x = torch.zeros(4, 2, 8)
    for bias, err in ((torch.zeros(7), ValueError), (torch.zeros(3, 8), ValueError),
                      (torch.zeros(8).bfloat16(), TypeError)):
        with pytest.raises(err):
            kda.layernorm_backward(x, x, bias=bias)
    with pytest.raises(ValueError, match="bias"):
        kda.layernorm_backward(x, x, torch.ones(8), bias=torch.zeros(2, 8))
