"""GPU: the global gradient norm, clipping in place and the clipped step.

Sums are compared with 64-bit sums of the same values: a sum of n squares in
doubles, in any order, is within n * 2^-53 of the exact one, and the norm's
conversion to fp32 adds half a step (2^-24).  Clipped gradients and the clipped
step are exact: one fp32 product by the coefficient that the norm call wrote,
rounded once, then the arithmetic of the step, which the oracle defines.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import sharded_state_amd as ss
from guards import Guarded
from parity import assert_bits_equal, dt_name, np_of

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(n, dtype, seed, sigma=1e-2):
    return (torch.randn(n, device="cuda", generator=_gen(seed)) * sigma).to(dtype)


def _exact(tensors):
    """(sum of squares, number of terms) in 64 bits."""
    return math.fsum(float(t.double().square().sum()) for t in tensors), sum(t.numel() for t in tensors)


def _check(gn, tensors, max_norm, what):
    q, n = _exact(tensors)
    torch.cuda.synchronize()
    tol = (2 * n + 4) * 2.0 ** -53               # both sums
    got = float(gn.sumsq)
    assert abs(got - q) <= tol * q, (what, got, q)
    norm = math.sqrt(q)
    assert abs(float(gn.norm) - norm) <= (2.0 ** -24 + tol) * norm, (what, float(gn.norm), norm)
    if max_norm is None:
        assert gn.coef is None
        return
    coef = min(1.0, max_norm / (norm + 1e-6))
    assert abs(float(gn.coef) - coef) <= (2.0 ** -24 + tol) * coef, (what, float(gn.coef), coef)


SIZES = [[1], [7], [4096], [8193, 1, 0, 4095], [100_003, 5, 70_000], [3] * 161, [0], [1 << 20, 65_537, 12]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
def test_norm_and_clip_of_a_list(dtype, sizes):
    print("case", dtype, sizes[:4], flush=True)
    ts = [_rand(n, dtype, 10 + k) for k, n in enumerate(sizes)]
    q, _ = _exact(ts)
    for max_norm in (None, 0.5 * math.sqrt(q), 2 * math.sqrt(q) + 1, 0.0):
        gn = ss.fsdp_grad_norm(ts, max_norm)
        _check(gn, ts, max_norm, (sizes[:4], max_norm))
        if max_norm is None:
            continue
        held = [Guarded(t.numel(), dtype, init=t) for t in ts]
        ss.fsdp_clip_grads([h.t for h in held], gn)
        for h, t in zip(held, ts):
            h.check("clip")
            want = (t.float().cpu() * gn.coef.cpu()).to(dtype)
            assert_bits_equal(np_of(h.t), np_of(want), "clipped")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 2, 3, 7])
def test_tensors_off_the_16_byte_grid(dtype, offset):
    es = torch.empty(0, dtype=dtype).element_size()
    print("case", dtype, offset, flush=True)
    ts = [_rand(n, dtype, k) for k, n in enumerate((20_001, 4096, 9))]
    held = [Guarded(t.numel(), dtype, offset=offset * es, init=t) for t in ts]
    gn = ss.fsdp_grad_norm([h.t for h in held], 0.1)
    _check(gn, ts, 0.1, offset)
    ss.fsdp_clip_grads([h.t for h in held], gn)
    for h, t in zip(held, ts):
        h.check("clip")
        assert_bits_equal(np_of(h.t), np_of((t.float().cpu() * gn.coef.cpu()).to(dtype)), "clipped")


def test_mixed_formats_and_the_same_bits_twice():
    ts = [_rand(n, DTYPES[k % 3], k) for k, n in enumerate([5, 70_001, 300, 1, 4097, 123_456, 64])]
    a, b = ss.fsdp_grad_norm(ts, 1.0), ss.fsdp_grad_norm(ts, 1.0)
    _check(a, ts, 1.0, "mixed")
    assert torch.equal(a.sumsq.view(torch.int64), b.sumsq.view(torch.int64))


def test_list_refusals():
    good, coef = torch.ones(8, device="cuda"), torch.ones(1, device="cuda")
    for bad, what in ((torch.ones(8), ValueError), (torch.ones(8, dtype=torch.int32, device="cuda"), TypeError),
                      (torch.ones(8, 8, device="cuda")[:, 1], ValueError), (None, TypeError),
                      (torch.ones(8, dtype=torch.float64, device="cuda"), TypeError)):
        with pytest.raises(what):
            ss.fsdp_grad_norm([good, bad])
        with pytest.raises(what):
            ss.fsdp_clip_grads([good, bad], coef)
    assert (good == 1).all()
    with pytest.raises(RuntimeError):
        ss.fsdp_clip_grads([good, good], coef)           # the same tensor twice


def test_extreme_values():
    """fp32 values whose squares overflow or vanish in fp32, infinities, NaN."""
    for v, n in ((3e38, 1000), (1e-30, 1000), (1e-45, 7)):
        t = torch.full((n,), v, device="cuda")
        gn = ss.fsdp_grad_norm([t], 1.0)
        want = float(t[0]) * math.sqrt(n)
        got = float(gn.norm)
        if want > 3.4028235e38:
            assert got == math.inf
        else:                                     # below the normal range a step is 2^-149
            assert abs(got - want) <= max(2.0 ** -23 * want, 2.0 ** -149)
        assert abs(float(gn.coef) - min(1.0, 1 / (want + 1e-6))) <= 2.0 ** -23
    t = torch.ones(5000, device="cuda")
    t[4321] = math.inf
    gn = ss.fsdp_grad_norm([t], 1.0)
    assert float(gn.norm) == math.inf and float(gn.coef) == 0.0
    ss.fsdp_clip_grads([t], gn)
    assert torch.isnan(t[4321]) and float(t.nansum()) == 0.0       # inf * 0, and zeros
    t = torch.ones(5000, device="cuda", dtype=torch.bfloat16)
    t[17] = math.nan
    gn = ss.fsdp_grad_norm([t, torch.full((3,), math.inf, device="cuda")], 1.0)
    assert math.isnan(float(gn.norm)) and math.isnan(float(gn.coef))
    ss.fsdp_clip_grads([t], gn)
    assert torch.isnan(t).all()


def test_more_than_2_to_the_31_elements():
    n = (1 << 31) + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-3:] = torch.tensor([3.0, 4.0, 12.0], dtype=torch.bfloat16, device="cuda")
    gn = ss.fsdp_grad_norm([t], 6.5)
    assert float(gn.sumsq) == 169.0 and float(gn.norm) == 13.0
    ss.fsdp_clip_grads([t], gn)
    assert t[-4:].tolist() == [0.0, 1.5, 2.0, 6.0] and float(t[:1000].abs().max()) == 0.0


UNITS = [
    (1, 0, torch.float32, True, [1000, 3]), (1, 0, torch.bfloat16, False, [4096 * 8 + 5]),
    (2, 1, torch.float16, True, [513, 100_000, 1]), (2, 0, torch.float16, False, [70_001]),
    (3, 2, torch.bfloat16, True, [4100, 8]), (4, 3, torch.bfloat16, False, [50_000, 64, 640]),
    (8, 5, torch.bfloat16, False, [65_536 + 24]), (8, 0, torch.float16, True, [2048] * 39),
    (5, 1, torch.float32, False, [777]), (8, 7, torch.float32, True, [12_345]),
]


def _units(world, dtype, sizes, seed=0):
    out = []
    for k, S in enumerate(sizes):
        pad = -(-world * S // 64) * 64
        rows = torch.zeros(world, pad, dtype=dtype, device="cuda")[:, :world * S]
        for q in range(world):
            rows[q].copy_(_rand(world * S, dtype, seed + 100 * k + q))
        out.append(list(rows))
    return out


@pytest.mark.parametrize("world,rank,dtype,fp32r,sizes", UNITS)
@pytest.mark.parametrize("store", [False, True])
def test_norm_of_units_is_that_of_the_reduce_scatter(world, rank, dtype, fp32r, sizes, store):
    print("case", world, rank, dtype, fp32r, len(sizes), store, flush=True)
    grads = _units(world, dtype, sizes)
    want = [ss.fsdp_reduce_scatter_local(g, rank, fp32r, shard_numel=S) for g, S in zip(grads, sizes)]
    held = [Guarded(S, w.dtype) for S, w in zip(sizes, want)]
    units = [dict(rank_grads=g, grad_shard=h.t) if store else dict(rank_grads=g, shard_numel=S)
             for g, h, S in zip(grads, held, sizes)]
    gn = ss.fsdp_grad_norm_units(units, rank, fp32r, 0.05)
    _check(gn, want, 0.05, "units")
    for h, w in zip(held, want):
        h.check("shard")
        if store:
            assert_bits_equal(np_of(h.t), np_of(w), "shard")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_16_bit_average_keeps_the_sign_of_zero(dtype):
    for world in (1, 2, 3, 4, 8):
        S = 1032
        grads = [torch.full((world * S,), -0.0, dtype=dtype, device="cuda") for _ in range(world)]
        out = torch.zeros(S, dtype=dtype, device="cuda")
        gn = ss.fsdp_grad_norm_units([dict(rank_grads=grads, grad_shard=out)], 0, False, 1.0)
        want = oracle.grad_average([np_of(g) for g in grads], 0, S, dt_name(dtype), False)
        got = np_of(out)
        assert np.array_equal(got, oracle.f32_to(np.asarray(want, dtype=np.float32), dt_name(dtype))
                              if np.asarray(want).dtype == np.float32 else want)
        assert (got == 0x8000).all() and float(gn.norm) == 0.0 and float(gn.coef) == 1.0


def test_units_off_the_16_byte_grid():
    S, world = 3001, 2
    held = [Guarded(world * S, torch.float16, offset=2 * (q + 1), init=_rand(world * S, torch.float16, q))
            for q in range(world)]
    grads = [h.t for h in held]
    want = ss.fsdp_reduce_scatter_local(grads, 1, False)
    out = Guarded(S, torch.float16, offset=6)
    gn = ss.fsdp_grad_norm_units([dict(rank_grads=grads, grad_shard=out.t)], 1, False)
    out.check("shard")
    assert_bits_equal(np_of(out.t), np_of(want), "shard")
    _check(gn, [want], None, "off the grid")


def test_combine_of_the_ranks():
    world, S = 4, 9001
    grads = _units(world, torch.bfloat16, [S])[0]
    shards = [ss.fsdp_reduce_scatter_local(grads, r, True) for r in range(world)]
    sums = torch.cat([ss.fsdp_grad_norm_units([dict(rank_grads=grads, shard_numel=S)], r, True).sumsq
                      for r in range(world)])
    gn = ss.fsdp_grad_norm_combine(sums, 0.25)
    _check(gn, shards, 0.25, "combine")
    none = ss.fsdp_grad_norm_combine(torch.empty(0, dtype=torch.float64, device="cuda"), 1.0)
    assert float(none.norm) == 0.0 and float(none.coef) == 1.0


def _step_units(world, rank, dtype, cdt, sizes, gather, seed=0, sdt=torch.float32):
    units = []
    for k, (g, S) in enumerate(zip(_units(world, dtype, sizes, seed), sizes)):
        u = dict(rank_grads=g, master=_rand(S, sdt, 7 + k, 0.02), exp_avg=_rand(S, sdt, 8 + k, 1e-3),
                 exp_avg_sq=_rand(S, sdt, 9 + k, 1e-3).abs())
        if gather:
            u["peer_shards"] = [None if q == rank else _rand(S, cdt, 50 + q) for q in range(world)]
            u["full"] = torch.zeros(world * S, dtype=cdt, device="cuda")
        elif sdt == torch.float32:
            u["compute_shard"] = torch.zeros(S, dtype=cdt, device="cuda")
        units.append(u)
    return units


@pytest.mark.parametrize("world,rank,dtype,fp32r,cdt,sizes,gather", [
    (2, 1, torch.float16, True, torch.float16, [5000, 700_001], True),
    (8, 2, torch.bfloat16, False, torch.bfloat16, [4096 + 8], True),
    (1, 0, torch.float32, True, torch.bfloat16, [1001], False),
    (3, 0, torch.float16, False, torch.float32, [999, 2048], False),
])
def test_clipped_step_matches_the_oracle(world, rank, dtype, fp32r, cdt, sizes, gather):
    print("case", world, dtype, fp32r, cdt, sizes, gather, flush=True)
    units = _step_units(world, rank, dtype, cdt, sizes, gather)
    before = [[np_of(u[k]).copy() for k in ("master", "exp_avg", "exp_avg_sq")] for u in units]
    avg = [ss.fsdp_reduce_scatter_local(u["rank_grads"], rank, fp32r, shard_numel=u["master"].numel()) for u in units]
    gn = ss.fsdp_grad_norm_units(units, rank, fp32r, 0.01)
    hp = ss.AdamWHP(step=3)
    call = ss.fsdp_step_units(units, rank, fp32r, hp, clip=gn)
    torch.cuda.synchronize()
    assert 0 < float(gn.coef) < 1 and call.hp.step == 3
    h = oracle.hp(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, 3)
    for u, (p, m, v), a in zip(units, before, avg):
        g = np_of(a.float().cpu() * gn.coef.cpu())
        _, comp = oracle.rank_step([g], 0, p, m, v, h, "f32", True, dt_name(cdt))
        for key, want in (("master", p), ("exp_avg", m), ("exp_avg_sq", v)):
            assert_bits_equal(np_of(u[key]), want, key)
        S = a.numel()
        own = u["full"][rank * S:(rank + 1) * S] if gather else u["compute_shard"]
        assert_bits_equal(np_of(own), comp, "compute")


@pytest.mark.parametrize("hp", [ss.OptimHP.sgd(momentum=0.9), ss.OptimHP.adamax(), ss.OptimHP.adadelta(),
                                ss.AdamWHP(step=2)], ids=["sgd", "adamax", "adadelta", "adamw"])
def test_a_coefficient_of_one_is_the_plain_step(hp):
    a, b = (_step_units(2, 0, torch.float16, torch.float16, [3000, 70_003], True) for _ in range(2))
    ss.fsdp_step_units(a, 0, True, hp)
    ss.fsdp_step_units(b, 0, True, hp, clip=torch.ones(1, device="cuda"))
    for x, y in zip(a, b):
        for key in ("master", "exp_avg", "exp_avg_sq", "full"):
            assert_bits_equal(np_of(y[key]), np_of(x[key]), key)


@pytest.mark.parametrize("offset", [1, 3])
@pytest.mark.parametrize("world,rank,dtype,fp32r,cdt,sdt,gather,hp", [
    (1, 0, torch.float16, True, torch.float16, torch.float32, True, ss.AdamWHP(step=2)),
    (2, 1, torch.bfloat16, True, torch.float32, torch.float32, True, ss.AdamWHP(step=2)),
    (3, 2, torch.float32, True, torch.bfloat16, torch.float32, True, ss.OptimHP.adadelta()),
    (4, 0, torch.float16, False, torch.float16, torch.float32, False, ss.OptimHP.sgd()),
    (6, 5, torch.bfloat16, False, torch.bfloat16, torch.float32, True, ss.OptimHP.sgd(momentum=0.9)),
    (8, 3, torch.bfloat16, True, torch.float16, torch.float32, True, ss.OptimHP.adamax()),
    (2, 0, torch.bfloat16, False, torch.bfloat16, torch.bfloat16, True, ss.AdamWHP(step=2)),
    (5, 1, torch.float16, False, torch.float16, torch.float16, True, ss.AdamWHP(step=2)),
])
def test_clipped_step_off_the_16_byte_grid(world, rank, dtype, fp32r, cdt, sdt, gather, hp, offset):
    """Units with buffers at odd offsets, beside one on the grid: a coefficient of 1
    gives the plain step's bits, in those places and nowhere else."""
    print("case", world, dtype, fp32r, cdt, sdt, gather, offset, flush=True)
    sizes = [511, 5003, 70_001, 4096]

    def make():
        units, guards = _step_units(world, rank, dtype, cdt, sizes, gather, sdt=sdt), []
        for u in units[:3]:
            for key in ("master", "exp_avg", "exp_avg_sq", "full", "compute_shard"):
                if u.get(key) is not None:
                    t = u[key]
                    g = Guarded(t.numel(), t.dtype, offset=offset * t.element_size(), init=t)
                    guards.append(g)
                    u[key] = g.t
        return units, guards

    (a, ga), (b, gb) = make(), make()
    ss.fsdp_step_units(a, rank, fp32r, hp)
    ss.fsdp_step_units(b, rank, fp32r, hp, clip=torch.ones(1, device="cuda"))
    for g in ga + gb:
        g.check("a buffer")
    for x, y in zip(a, b):
        for key in ("master", "exp_avg", "exp_avg_sq", "full", "compute_shard"):
            if x.get(key) is not None:
                assert_bits_equal(np_of(y[key]), np_of(x[key]), key)


def test_clipped_step_with_16_bit_state():
    a, b = (_step_units(2, 1, torch.bfloat16, torch.bfloat16, [6000], True, sdt=torch.bfloat16) for _ in range(2))
    coef = torch.tensor([0.5], device="cuda")
    half = [dict(u, rank_grads=[g * 0.5 for g in u["rank_grads"]]) for u in b]     # exact in bf16
    ss.fsdp_step_units(a, 1, True, ss.AdamWHP(step=2), clip=coef)
    ss.fsdp_step_units(half, 1, True, ss.AdamWHP(step=2))
    for x, y in zip(a, b):
        for key in ("master", "exp_avg", "exp_avg_sq", "full"):
            assert_bits_equal(np_of(x[key]), np_of(y[key]), key)


def test_norm_and_clipped_step_on_another_stream_and_replayed():
    """Norm and step captured together: every replay reads the coefficient that
    its own norm wrote."""
    rank, fp32r, hp = 1, True, ss.AdamWHP(step=5)
    a = _step_units(2, rank, torch.float16, torch.float16, [4099, 70_000], True)
    b = [dict(u, master=u["master"].clone(), exp_avg=u["exp_avg"].clone(), exp_avg_sq=u["exp_avg_sq"].clone(),
              full=u["full"].clone()) for u in a]
    gn_a, gn_b = ss.GradNorm(), ss.GradNorm()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ss.fsdp_grad_norm_units(a, rank, fp32r, 0.1, out=gn_a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ss.fsdp_grad_norm_units(b, rank, fp32r, 0.1, out=gn_b)
    assert torch.equal(gn_a.sumsq, gn_b.sumsq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.fsdp_grad_norm_units(a, rank, fp32r, 0.1, out=gn_a)
        ss.prepare_step_units(a, rank, fp32r, hp, clip=gn_a)()
    torch.cuda.synchronize()
    for replay in range(3):
        for u, w in zip(a, b):                   # other gradients for every replay
            for g, h in zip(u["rank_grads"], w["rank_grads"]):
                g.mul_(1.5)
                assert g.data_ptr() == h.data_ptr()      # the two tables share their gradients
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ss.fsdp_grad_norm_units(b, rank, fp32r, 0.1, out=gn_b)
        ss.fsdp_step_units(b, rank, fp32r, hp, clip=gn_b)
        torch.cuda.synchronize()
        assert torch.equal(gn_a.norm, gn_b.norm) and torch.equal(gn_a.coef, gn_b.coef), replay
        for u, w in zip(a, b):
            for key in ("master", "exp_avg", "exp_avg_sq", "full"):
                assert_bits_equal(np_of(u[key]), np_of(w[key]), "replay %d %s" % (replay, key))


def test_unit_config_norm_and_step():
    cfg = ss.from_fairseq(2, 1, fp16=True, fp32_reduce_scatter=True, no_reshard_after_forward=True)
    a, b = (_step_units(2, 1, torch.float16, torch.float16, [3000], True) for _ in range(2))
    hp = ss.AdamWHP(step=1)
    cfg.step(a, hp, clip=cfg.grad_norm(a, 0.02))
    ss.fsdp_step_units(b, 1, True, hp, clip=ss.fsdp_grad_norm_units(b, 1, True, 0.02))
    assert_bits_equal(np_of(a[0]["master"]), np_of(b[0]["master"]), "master")
