"""GPU: 4-bit products of more tiles than one launch takes."""
import pytest
import torch

import sharded_state_amd as ss

pytestmark = pytest.mark.gpu


@pytest.fixture
def room():
    yield
    torch.cuda.empty_cache()


def test_one_token_through_more_rows_than_a_launch(room):
    n, k = (1 << 27) + 40, 32
    codes = torch.full((n, 16), 0x22, dtype=torch.uint8, device="cuda")          # ones
    scales = torch.full((n, 1), 127, dtype=torch.uint8, device="cuda")
    marks = [0, (1 << 26) - 1, 1 << 26, (1 << 27) - 17, (1 << 27) - 16, 1 << 27, n - 1]
    for i, r in enumerate(marks):
        scales[r] = 128 + i
    y = ss.fsdp_mx4_linear(torch.ones(1, k, device="cuda"), ss.Mx4(codes, scales, k))
    want = torch.full((1, n), 32.0, device="cuda")
    for i, r in enumerate(marks):
        want[0, r] = 64.0 * 2 ** i
    assert torch.equal(y, want)


def test_product_of_more_tiles_than_a_launch(room):
    n, k = (1 << 31) + 300, 32
    codes = torch.full((n, 16), 0x22, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, 1), 127, dtype=torch.uint8, device="cuda")
    marks = [0, (1 << 30) - 1, 1 << 30, (1 << 31) - 257, (1 << 31) - 256, 1 << 31, n - 1]
    for i, r in enumerate(marks):
        scales[r] = 128 + i
    long = ss.Mx4(codes, scales, k)
    one = ss.Mx4(torch.full((1, 16), 0x22, dtype=torch.uint8, device="cuda"),
                 torch.full((1, 1), 127, dtype=torch.uint8, device="cuda"), k)
    for a, b in ((long, one), (one, long)):
        y = ss.fsdp_mx4_matmul(a, b).view(-1)
        for i, r in enumerate(marks):
            assert float(y[r]) == 64.0 * 2 ** i, (a.rows, r)
            y[r] = 32.0
        assert bool((y == 32).all()), a.rows
        del y
