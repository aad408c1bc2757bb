"""The norm over units refuses sizes that contradict each other."""
import pytest
import torch

import sharded_state_amd as ss


@pytest.mark.parametrize("unit", [dict(master=torch.zeros(8)), dict(shard_numel=8),
                                  dict(master=torch.zeros(6), shard_numel=6)])
def test_a_gradient_shard_of_another_size_than_the_unit_is_refused(unit):
    unit = dict(unit, rank_grads=[torch.zeros(16)] * 2, grad_shard=torch.zeros(6))
    if "master" in unit and "shard_numel" in unit:
        unit["shard_numel"] = 8
    with pytest.raises(ValueError, match="units\\[0\\].*6.*8|units\\[0\\].*8.*6"):
        ss.fsdp_grad_norm_units([unit], 0, True)
