"""Results that are written into tensors of the caller's count as changes of them, and
a call that is refused changes nothing.  Host memory: what hands the addresses to the
library is put aside."""
import pytest
import torch

import sharded_state_amd as ss
from sharded_state_amd import fp8, mx4, rms


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    def matrix(t, name):
        return (*t.shape, t.stride(0)) if t.dim() == 2 else (1, t.shape[0], t.shape[0])

    for module in (fp8, mx4, rms):
        monkeypatch.setattr(module, "_matrix", matrix)
        monkeypatch.setattr(module, "_issue", lambda *args: None)
    monkeypatch.setattr(fp8, "_operand", lambda t, name: t)


def _versions(*tensors):
    return [t._version for t in tensors]


def test_norm_and_its_gradients():
    x, res, y, w = *(torch.zeros(3, 64) for _ in range(3)), torch.ones(64)
    before = _versions(x, res, y, w)
    with torch.no_grad():
        o = ss.fsdp_rms_norm_fp8(x, w, res, y=y)
        assert o.y is y and _versions(x, res, y, w) == [before[0], before[1], before[2] + 1, before[3]]
        ss.fsdp_rms_norm_fp8(x, w, res, h=res)
        ss.fsdp_rms_norm_fp8(x, w, res, h=x)
    assert _versions(x, res, w) == [before[0] + 1, before[1] + 1, before[3]]
    flat = torch.zeros(100)
    rstd = torch.ones(3)
    before = _versions(x, res, w, rstd, flat)
    ss.fsdp_rms_norm_grads(x, res, w, rstd, dh=y, dx=x, dw=flat[36:])
    assert _versions(x, res, w, rstd, flat) == [before[0] + 1, *before[1:4], before[4] + 1]
    ss.fsdp_rms_norm_grads(x, res, w, rstd, dx=False, dw=False)
    with pytest.raises(ValueError):
        ss.fsdp_rms_norm_grads(x, res, w, rstd, dx=y, dw=flat)
    assert _versions(x, y, flat) == [before[0] + 1, 1, before[4] + 1]


@pytest.mark.parametrize("blocks", [ss.Fp8, ss.Mx4])
def test_products_and_their_gradients(blocks):
    matmul, linear, grads = ((ss.fsdp_fp8_matmul, ss.fsdp_fp8_linear, ss.fsdp_fp8_linear_grads) if blocks is ss.Fp8 else
                             (ss.fsdp_mx4_matmul, ss.fsdp_mx4_linear, ss.fsdp_mx4_linear_grads))
    w, wt = blocks.empty(96, 64, "cpu"), blocks.empty(64, 96, "cpu")
    x, dy, dx, dw, y = torch.zeros(3, 64), torch.zeros(3, 96), torch.zeros(3, 64), torch.zeros(96, 64), torch.zeros(3, 96)
    linear(x, w, y)
    assert _versions(x, y) == [0, 1]
    if blocks is ss.Fp8:                                     # the 4-bit product looks at its operands' memory
        matmul(blocks.empty(3, 64, "cpu"), w, y)
        linear(blocks.empty(3, 64, "cpu"), w, y)
        assert y._version == 3
    grads(dy, x, wt, dx=dx, dw=dw)
    assert _versions(dy, x, dx, dw) == [0, 0, 1, 1]
    grads(dy, x, wt, dx=dx, dw=False)
    grads(dy, x, wt)
    assert _versions(dy, x, dx, dw) == [0, 0, 2, 1]


def test_a_graph_that_saved_the_residual_refuses_its_backward():
    a = torch.ones(3, 64, requires_grad=True)
    res = a * 2
    loss = res.square().sum()                                # saves res
    ss.fsdp_rms_norm_fp8(torch.ones(3, 64), torch.ones(64), res.detach(), h=res.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_rstd_of_no_features_is_not_what_memory_held(monkeypatch):
    """Its mean is one of nothing: NaN."""
    monkeypatch.setattr(rms, "_vector", lambda n, dtype, device, stream: torch.full((n,), 7.0, dtype=dtype))
    o = ss.fsdp_rms_norm_fp8(torch.zeros(3, 0), torch.zeros(0))
    assert o.rstd.shape == (3,) and o.rstd.isnan().all()
