"""GPU: the combine of as many sums of squares as its count can say, whose last
indexes lie within a workgroup's pass of 2^31."""
import pytest
import torch

import sharded_state_amd as ss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [4096, 4097, (1 << 31) - 4096, (1 << 31) - 1])
def test_combine_up_to_the_largest_count(n):
    print("case", n, flush=True)
    sums = torch.zeros(n, dtype=torch.float64, device="cuda")
    sums[0], sums[n // 2], sums[n - 1025], sums[n - 1] = 9.0, 16.0, 144.0, 3600.0
    gn = ss.fsdp_grad_norm_combine(sums, 10.0)
    assert float(gn.sumsq) == 3769.0
    assert float(gn.norm) == float(torch.tensor(3769.0, dtype=torch.float64).sqrt().float())
    del sums
    torch.cuda.empty_cache()
