"""GPU: averages of -0 reduced in 16 bits keep their sign through the
reduce-scatter, the norm over units and the step, as the oracle has it, on the
vector path, in the tail and off the 16-byte grid."""
import numpy as np
import pytest
import torch

import oracle
import sharded_state_amd as ss
from parity import assert_bits_equal, dt_name, np_of

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]


def _grads(world, S, dtype, off=0):
    """-0 at every third place, small values of both signs elsewhere (some of
    whose averages round to -0)."""
    out = []
    for q in range(world):
        g = torch.Generator(device="cuda")
        g.manual_seed(q)
        t = torch.randn(world * S, device="cuda", generator=g).to(dtype)
        t[::3] = -0.0
        t[1::7] = -torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        buf = torch.empty(world * S + off, dtype=dtype, device="cuda")
        buf[off:].copy_(t)
        out.append(buf[off:])
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("world", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("S,off", [(1032, 0), (4096, 0), (1003, 1)])
def test_reduce_scatter_and_norm_over_units(world, dtype, S, off):
    print("case", world, dtype, S, off, flush=True)
    grads = _grads(world, S, dtype, off)
    rank = world - 1
    want = oracle.grad_average([np_of(g) for g in grads], rank * S, S, dt_name(dtype), False)
    # a third of the places without their seventh part: 2/7 of them, but for the block's ends
    assert (want == 0x8000).sum() > S // 4
    got = ss.fsdp_reduce_scatter_local(grads, rank, False, shard_numel=S)
    assert_bits_equal(np_of(got), want, "reduce-scatter")
    kept = torch.empty(S + off, dtype=dtype, device="cuda")[off:]
    ss.fsdp_grad_norm_units([dict(rank_grads=grads, grad_shard=kept)], rank, False)
    assert_bits_equal(np_of(kept), np_of(got), "norm over units")


@pytest.mark.parametrize("world", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("S,off", [(1032, 0), (1003, 1)])
@pytest.mark.parametrize("clip", [False, True])
def test_step_whose_first_moment_is_minus_zero(world, S, off, clip):
    """m = beta1 * -0 + (1 - beta1) * -0 is -0 only where the average is."""
    print("case", world, S, off, clip, flush=True)
    grads = _grads(world, S, torch.float16, off)
    rank, hp = 0, ss.AdamWHP(step=2)
    state = [torch.empty(S + off, device="cuda")[off:] for _ in range(3)]
    state[0].normal_()
    state[1].fill_(-0.0)
    state[2].zero_()
    want = [np_of(t).copy() for t in state]
    oracle.rank_step([np_of(g) for g in grads], rank, *want,
                     oracle.hp(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, 2), "f16", False, "f16")
    unit = dict(master=state[0], exp_avg=state[1], exp_avg_sq=state[2], rank_grads=grads,
                compute_shard=torch.empty(S, dtype=torch.float16, device="cuda"))
    ss.fsdp_step_units([unit], rank, False, hp, clip=torch.ones(1, device="cuda") if clip else None)
    torch.cuda.synchronize()
    assert np.signbit(want[1][want[1] == 0]).any()
    for t, w, what in zip(state, want, ("master", "exp_avg", "exp_avg_sq")):
        assert_bits_equal(np_of(t), w, what)
