"""GPU: a coefficient does not outlive the norm that it belongs to.  A norm taken
without a bound into a GradNorm whose coefficient a prepared or captured step reads
leaves there the coefficient of no clipping, by the formula with the largest bound:
1, or 0 and NaN where the norm is infinite or NaN."""
import math

import pytest
import torch

import sharded_state_amd as ss
from parity import assert_bits_equal, np_of

pytestmark = pytest.mark.gpu

KEYS = ("master", "exp_avg", "exp_avg_sq", "compute_shard")


def _unit(S=5000, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(n, sigma):
        return torch.randn(n, device="cuda", generator=g) * sigma

    return dict(rank_grads=[rand(2 * S, 1e-2).half() for _ in range(2)], master=rand(S, 0.02), exp_avg=rand(S, 1e-3),
                exp_avg_sq=rand(S, 1e-3).abs(), compute_shard=torch.zeros(S, dtype=torch.float16, device="cuda"))


def _takes(unit):
    """The norm calls of every kind, as functions of (max_norm, out)."""
    one, many = torch.full((7,), 3.0, device="cuda"), [torch.ones(70_001, device="cuda").bfloat16()] * 2
    sums = torch.tensor([9.0, 16.0], dtype=torch.float64, device="cuda")
    return (lambda b, o: ss.fsdp_grad_norm([one], b, out=o), lambda b, o: ss.fsdp_grad_norm(many, b, out=o),
            lambda b, o: ss.fsdp_grad_norm_units([unit], 1, True, b, out=o),
            lambda b, o: ss.fsdp_grad_norm_combine(sums, b, out=o))


@pytest.mark.parametrize("kind", range(4), ids=["one chunk", "list", "units", "combine"])
def test_a_norm_without_a_bound_sets_the_coefficient_to_one(kind):
    take = _takes(_unit())[kind]
    gn = take(1e-3, ss.GradNorm())
    coef = gn.coef
    assert 0 < float(coef) < 1
    take(None, gn)
    assert gn.coef is None and float(coef) == 1.0
    take(1e-3, gn)
    assert 0 < float(coef) < 1 and gn.coef is not None


def test_by_the_formula_where_the_norm_is_not_finite():
    gn = ss.fsdp_grad_norm([torch.ones(5, device="cuda")], 0.5)
    coef = gn.coef
    for bad, want in ((math.inf, 0.0), (math.nan, math.nan), (1.0, 1.0), (3e38, 1.0), (0.0, 1.0)):
        ss.fsdp_grad_norm([torch.tensor([bad, 1.0], device="cuda")], out=gn)
        assert float(coef) == want or (math.isnan(want) and math.isnan(float(coef))), (bad, float(coef))


def test_a_prepared_and_a_captured_step_after_a_norm_without_a_bound():
    a, b, c = _unit(), _unit(), _unit()
    hp = ss.AdamWHP(step=2)
    gn = ss.fsdp_grad_norm_units([a], 1, True, 1e-3)
    call = ss.prepare_step_units([a], 1, True, hp, clip=gn)
    captured = ss.prepare_step_units([c], 1, True, hp, clip=gn)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    ss.fsdp_grad_norm_units([a], 1, True, out=gn)            # this iteration clips nothing
    call()
    graph.replay()
    ss.fsdp_step_units([b], 1, True, hp)
    torch.cuda.synchronize()
    for key in KEYS:
        assert_bits_equal(np_of(a[key]), np_of(b[key]), "prepared, " + key)
        assert_bits_equal(np_of(c[key]), np_of(b[key]), "captured, " + key)
