"""GPU: 4-bit blocks along the columns of more tiles than one launch takes."""
import pytest
import torch

import sharded_state_amd as ss

pytestmark = pytest.mark.gpu


@pytest.fixture
def room():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_columns_of_more_tiles_than_a_launch(room, dtype):
    n = (1 << 30) + 69
    x = torch.arange(n, device="cuda", dtype=torch.int32).remainder_(1021).sub_(500).to(dtype)
    flat = ss.fsdp_mx4_quantize(x)                       # one row
    tall = ss.fsdp_mx4_quantize(x.view(n, 1), form="columns")
    assert torch.equal(tall.codes, flat.codes) and torch.equal(tall.scales, flat.scales)
    del tall, flat
    each = ss.fsdp_mx4_quantize(x.view(n, 1))            # every element a block
    wide = ss.fsdp_mx4_quantize(x.view(1, n), form="columns")
    assert torch.equal(wide.codes, each.codes) and torch.equal(wide.scales, each.scales)
    del wide
    rows, cols = ss.fsdp_mx4_quantize(x.view(n, 1), form="both")
    assert torch.equal(rows.codes, each.codes) and torch.equal(rows.scales, each.scales)
    del rows, each
    flat = ss.fsdp_mx4_quantize(x)
    assert torch.equal(cols.codes, flat.codes) and torch.equal(cols.scales, flat.scales)


def test_gradient_of_a_weight_with_more_rows_than_a_launch(room):
    """dw of one token: dy's columns are more tiles than a launch takes."""
    n, k = (1 << 30) + 69, 2
    dy = torch.arange(n, device="cuda", dtype=torch.int32).remainder_(3).to(torch.bfloat16).view(1, n)
    x = torch.tensor([[1.0, -2.0]], device="cuda", dtype=torch.bfloat16)
    wt = ss.Mx4.empty(k, n)                              # not read: dx is not wanted
    dw = ss.fsdp_mx4_linear_grads(dy, x, wt, dx=False)[1]
    assert torch.equal(dw[:, 0], dy[0]) and torch.equal(dw[:, 1], -2 * dy[0])
