"""Inputs with a forward-mode tangent, which the outputs would lose, are refused; the
same inputs without one pass that check."""
import pytest
import torch
from torch.autograd import forward_ad

import sharded_state_amd as ss
from sharded_state_amd import fp8


def _calls():
    w8, t8 = ss.Fp8.empty(96, 64, "cpu"), ss.Fp8.empty(64, 96, "cpu")
    w4, t4 = ss.Mx4.empty(96, 64, "cpu"), ss.Mx4.empty(64, 96, "cpu")
    x, dy, w, rstd = torch.zeros(3, 64), torch.zeros(3, 96), torch.ones(64), torch.ones(3)
    return [(lambda x: ss.fsdp_fp8_linear(x, w8), [x]), (lambda x: ss.fsdp_mx4_linear(x, w4), [x]),
            (lambda dy, x: ss.fsdp_fp8_linear_grads(dy, x, t8), [dy, x]),
            (lambda dy, x: ss.fsdp_mx4_linear_grads(dy, x, t4), [dy, x]),
            (lambda x, w, r: ss.fsdp_rms_norm_fp8(x, w, r), [x, w, x]),
            (lambda dy, h, w, r, dh: ss.fsdp_rms_norm_grads(dy, h, w, r, dh=dh), [x, x, w, rstd, x])]


@pytest.mark.parametrize("call", range(6))
def test_tangents_are_refused(call, monkeypatch):
    monkeypatch.setattr(fp8, "_operand", lambda t, name: t)          # the 8-bit weights are in host memory too
    f, inputs = _calls()[call]
    with forward_ad.dual_level():
        for i, t in enumerate(inputs):
            given = list(inputs)
            given[i] = forward_ad.make_dual(t, torch.ones_like(t))
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                f(*given)
            given[i] = forward_ad.unpack_dual(given[i]).primal
            with pytest.raises(ValueError, match="device"):          # as far as the next check: host memory
                f(*given)
    with pytest.raises(ValueError, match="device"):
        f(*inputs)
