"""GPU: column slices of one buffer as x and y, dy and dx, dx and dw."""
import pytest
import torch

import sharded_state_amd as ss
from mx4_check import assert_equal, whole, whole_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(2, 65, 96), (16, 200, 33), (40, 64, 96), (300, 261, 130)])
def test_column_slices_of_one_buffer(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    x, w, dy = whole((m, k), 1, "cuda"), whole((n, k), 2, "cuda"), whole((m, n), 3, "cuda")
    both = torch.full((m, k + n + 1), 7.0, dtype=dtype, device="cuda")
    both[:, :k] = x
    ss.fsdp_mx4_linear(both[:, :k], ss.fsdp_mx4_quantize(w), both[:, k:k + n])
    assert_equal(both[:, k:k + n], whole_product(x, w, dtype), "y beside x")
    assert_equal(both[:, :k], x.to(dtype).cpu(), "x")
    assert (both[:, k + n:] == 7).all()
    wt = ss.fsdp_mx4_quantize(w, form="columns")
    rows = max(m, n)
    every = torch.full((rows, n + 3 * k + 2), 7.0, dtype=dtype, device="cuda")
    every[:m, :n], every[:m, n:n + k] = dy, x
    dx, dw = every[:m, n + k:n + 2 * k], every[:n, n + 2 * k:n + 3 * k]
    ss.fsdp_mx4_linear_grads(every[:m, :n], every[:m, n:n + k], wt, dx=dx, dw=dw)
    assert_equal(dx, whole_product(dy, w.T, dtype), "dx")
    assert_equal(dw, whole_product(dy.T, x.T, dtype), "dw")
    assert_equal(every[:m, :n], dy.to(dtype).cpu(), "dy")
    assert (every[:, n + 3 * k:] == 7).all()
