"""GPU: results written into tensors of the caller's count as changes of them, also
where the call is captured."""
import pytest
import torch

import sharded_state_amd as ss

pytestmark = pytest.mark.gpu


def _rand(*shape):
    return torch.randn(shape, device="cuda")


@pytest.mark.parametrize("captured", [False, True])
def test_given_tensors_count_as_changed(captured):
    x, res, w = _rand(4, 256), _rand(4, 256), torch.ones(256, device="cuda")
    lin, t = ss.fsdp_fp8_quantize(_rand(384, 256), form="both", tile=True)
    lin4, t4 = ss.fsdp_mx4_quantize(_rand(384, 256), form="both")
    y, dy, dx, flat = _rand(4, 384), _rand(4, 384), _rand(4, 256), torch.zeros(1000 + 384 * 256, device="cuda")
    dw = flat[1000:].view(384, 256)

    def calls():
        o = ss.fsdp_rms_norm_fp8(x, w, res, h=res)
        ss.fsdp_fp8_linear(o.q, lin, y)
        ss.fsdp_fp8_linear(x, lin, y)
        ss.fsdp_fp8_linear_grads(dy, x, t, dx=dx, dw=dw)
        ss.fsdp_rms_norm_grads(dx, res, w, o.rstd, dx=dx)
        ss.fsdp_mx4_linear(x, lin4, y)
        ss.fsdp_mx4_matmul(ss.fsdp_mx4_quantize(x), lin4, y)
        ss.fsdp_mx4_linear_grads(dy, x, t4, dx=dx, dw=dw)

    tensors = (x, w, dy, res, y, dx, flat)
    before = [a._version for a in tensors]
    if captured:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            calls()
    else:
        calls()
    torch.cuda.synchronize()
    assert [a._version - b for a, b in zip(tensors, before)] == [0, 0, 0, 1, 4, 3, 2]


def test_a_graph_that_saved_the_residual_refuses_its_backward():
    a = _rand(3, 64).requires_grad_()
    res = a * 2
    loss = res.square().sum()
    held = res.detach()
    ss.fsdp_rms_norm_fp8(_rand(3, 64), torch.ones(64, device="cuda"), held, h=held)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
