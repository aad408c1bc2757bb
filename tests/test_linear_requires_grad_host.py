"""The 4-bit linear refuses an x whose gradient would silently be lost."""
import pytest
import torch

import sharded_state_amd as ss


def test_linear_refuses_an_x_whose_gradient_would_be_lost():
    w = ss.Mx4.empty(4, 64, "cpu")
    x = torch.zeros(2, 64, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        ss.fsdp_mx4_linear(x, w)
    for ok in (x.detach(), x):                       # as far as the next check: host memory
        with torch.no_grad(), pytest.raises(ValueError, match="device"):
            ss.fsdp_mx4_linear(ok, w)
