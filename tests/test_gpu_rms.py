"""GPU: the root-mean-square norm with the residual's addition and 8-bit output, and
its gradients.

Tolerances count roundings of half a step (u = 2^-24 in fp32).  h is the fp32 sum
rounded to its type: exact.  rstd comes from 64-bit sums and is rounded once: u of
its value (and the 64-bit arithmetic's 2^-50, far under the next).  y is a 64-bit
product, rounded once where it is returned in fp32.  The blocks are those of the
64-bit product, bit for bit (not of the fp32 y: rounding that once more takes 1 code
in 2^20 to a neighbour, where the first rounding ends on a tie).
dx = rstd * (g - h * f) + dh: g one rounding, f one more than g's, their products and
sums one each: 6 u of rstd * (|g| + |h| F) + |dh|, F = rstd^2 sum|g h| / d, then the
type's half step.  dw: two roundings a term and one an addition, in any order:
(m + 2) u of the sum of magnitudes, then the type's half step.
"""
import math

import numpy as np
import pytest
import torch

import fp8_ref
import sharded_state_amd as ss
from guards import Guarded
from mx4_check import assert_within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
SIZES = [(1, 1), (1, 8), (3, 7), (2, 100), (5, 127), (3, 129), (4, 511), (3, 512), (9, 1000), (2, 1024), (3, 1025),
         (33, 1600), (5, 2049), (2, 4097), (7, 5120), (2, 6145), (2, 8192), (3, 12_001), (2, 20_001), (1, 32_768),
         (2100, 40), (1300, 1100)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(shape, dtype=torch.float32, seed=0, sigma=1.0):
    return (torch.randn(shape, device="cuda", generator=_gen(seed)) * sigma).to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def _half(dtype):
    return torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _same_blocks(q, x):
    codes, scales = fp8_ref.quantize(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales), "scales"
    assert np.array_equal(q.codes.cpu().numpy(), codes), "codes"


def _check_norm(o, x, w, res, eps):
    """Checks an RmsNorm with a float32 y."""
    if res is None:
        assert o.h is x
    else:
        want = (x.cpu().float() + res.cpu().float()).to(res.dtype)
        assert torch.equal(_bits(o.h.cpu()), _bits(want)), "h"
    h, W = _f64(o.h), _f64(w)
    r = 1 / np.sqrt((h ** 2).sum(axis=1) / h.shape[1] + eps)
    assert_within(_f64(o.rstd), r, r * U * (1 + 2.0 ** -20), "rstd")
    y = h * r[:, None] * W
    assert_within(_f64(o.y), y, U * np.abs(y) * (1 + 2.0 ** -20) + 2.0 ** -149, "y")
    _same_blocks(o.q, y)


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("xt,ht", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float16, torch.float16), (torch.float32, torch.float32),
                                   (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float16)])
def test_norm(m, d, xt, ht):
    print("case", m, d, xt, ht, flush=True)
    size = torch.logspace(-2, 2, m, device="cuda")[:, None] if m > 1 else 1.0
    x, res = (_rand((m, d), sigma=1.0, seed=1) * size).to(xt), (_rand((m, d), sigma=2.0, seed=2) * size).to(ht)
    w = (1 + _rand((d,), sigma=0.2, seed=3)).to(DTYPES[(m + d) % 3])
    for eps in (1e-5, 0.0):
        o = ss.fsdp_rms_norm_fp8(x, w, res, eps=eps, y=torch.empty((m, d), device="cuda"))
        _check_norm(o, x, w, res, eps)
    alone = ss.fsdp_rms_norm_fp8(x, w, eps=1e-5, y=torch.empty((m, d), device="cuda"))
    _check_norm(alone, x, w, None, 1e-5)
    short = ss.fsdp_rms_norm_fp8(x, w, res, eps=1e-5)
    o = ss.fsdp_rms_norm_fp8(x, w, res, eps=1e-5, y=True)
    assert short.y is None and o.y.dtype == xt
    assert torch.equal(short.q.codes, o.q.codes) and torch.equal(short.q.scales, o.q.scales)
    y = ss.fsdp_rms_norm_fp8(x, w, res, eps=1e-5, y=torch.empty((m, d), device="cuda")).y
    assert torch.equal(_bits(o.y), _bits(y.to(xt)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,d", [(5, 77), (3, 1601), (4, 2050), (3, 8191), (2, 9001)])
def test_norm_of_strided_rows_at_any_alignment(m, d, dtype):
    """Rows with gaps, off the 16-byte grid, a weight in the middle of a flat unit; nothing else is written."""
    print("case", m, d, dtype, flush=True)
    es = torch.empty(0, dtype=dtype).element_size()
    for pad, off in ((3, 1), (8, 5)):
        ld = d + pad
        n = (m - 1) * ld + d
        held = {k: Guarded(n, dtype, offset=off * es, init=_rand((n,), dtype, i)) for i, k in enumerate("xr")}
        outs = {k: Guarded(n, dtype, offset=off * es) for k in "hy"}
        rows = {k: torch.as_strided(g.t, (m, d), (ld, 1)) for k, g in {**held, **outs}.items()}
        flat = _rand((d + 11,), dtype, 7)
        w = flat[11:]
        nb = -(-d // 128)
        codes, scales = Guarded(m * nb * 128, torch.uint8), Guarded(m * nb, torch.uint8, offset=1)
        q = ss.Fp8(codes.t.view(m, -1), scales.t.view(m, -1), d)
        o = ss.fsdp_rms_norm_fp8(rows["x"], w, rows["r"], out=q, h=rows["h"], y=rows["y"])
        for k, g in {**held, **outs, "codes": codes, "scales": scales}.items():
            g.check(k)
        assert o.q is q and o.h is rows["h"] and o.y is rows["y"]
        for k in "hy":
            gap = torch.as_strided(outs[k].t, (m - 1, pad), (ld, 1), outs[k].t.storage_offset() + d)
            assert (gap.contiguous().view(torch.uint8) == 0xA5).all(), k
        plain = ss.fsdp_rms_norm_fp8(rows["x"].contiguous(), w.clone(), rows["r"].contiguous(), y=True)
        assert torch.equal(_bits(plain.h), _bits(o.h)) and torch.equal(_bits(plain.y), _bits(o.y))
        assert torch.equal(plain.q.codes, q.codes) and torch.equal(plain.q.scales, q.scales)
        assert torch.equal(plain.rstd, o.rstd)
        # in place: h the residual, then h the x
        for k in "rx":
            keep = rows[k].clone()
            again = ss.fsdp_rms_norm_fp8(rows["x"], w, rows["r"], h=rows[k])
            assert again.h is rows[k] and torch.equal(_bits(again.h), _bits(plain.h))
            assert torch.equal(again.q.codes, q.codes)
            held[k].check(k)
            rows[k].copy_(keep)


def test_norm_of_zeros_and_of_values_that_are_not_finite():
    d = 300
    x = torch.zeros((6, d), device="cuda")
    x[1, 5], x[2, 200], x[3, 0] = math.inf, math.nan, -math.inf
    x[4] = 3e38
    x[5] = 1e-30
    w = torch.ones(d, device="cuda")
    o = ss.fsdp_rms_norm_fp8(x, w, eps=1e-6, y=True)
    assert not o.y[0].any() and o.rstd[0] == float(np.float32(1 / math.sqrt(1e-6)))
    # an infinite row: rstd 0, so zeros and infinity * 0; a NaN takes the whole row
    assert o.rstd[1] == 0 and torch.isnan(o.y[1]).nonzero().tolist() == [[5]]
    assert o.q.scales[1].tolist() == [255, 1, 1] and o.q.scales[3].tolist() == [255, 1, 1]
    assert torch.isnan(o.y[2]).all() and o.q.scales[2].tolist() == [255] * 3
    # squares that fp32 does not hold: 3e38 and 1e-30 (with no eps) are still normed to 1
    assert abs(float(o.y[4, 7]) - 1) <= 2.0 ** -20          # rstd is a subnormal of 20 bits
    o = ss.fsdp_rms_norm_fp8(x[5:], w, eps=0.0, y=True)
    assert abs(float(o.y[0, 9]) - 1) <= 4 * U
    # without eps a row of zeros is 0 * infinity
    assert torch.isnan(ss.fsdp_rms_norm_fp8(x[:1], w, eps=0.0, y=True).y).all()


def _check_grads(dx, dw, dy, h, w, rstd, dh):
    DY, H, W, R = _f64(dy), _f64(h), _f64(w), _f64(rstd)[:, None]
    m, d = DY.shape
    g = DY * W
    f = R ** 2 * (g * H).sum(axis=1, keepdims=True) / d
    F = R ** 2 * np.abs(g * H).sum(axis=1, keepdims=True) / d
    E = 0.0 if dh is None else _f64(dh)
    if dx is not None:
        want = R * (g - H * f) + E
        half, tiny = _half(dx.dtype)
        room = R * (np.abs(g) + np.abs(H) * F) + np.abs(E)
        assert_within(_f64(dx), want, 6 * U * room * (1 + half) + half * np.abs(want) + tiny + 2.0 ** -140, "dx")
    if dw is not None:
        terms = DY * (H * R)
        want = terms.sum(axis=0)
        half, tiny = _half(dw.dtype)
        assert_within(_f64(dw), want, (m + 2) * U * np.abs(terms).sum(axis=0) * (1 + half) + half * np.abs(want) + tiny, "dw")


@pytest.mark.parametrize("m,d", SIZES + [(5000, 129), (1025, 2050)])
@pytest.mark.parametrize("yt,ht", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                   (torch.float16, torch.float16), (torch.float32, torch.float32),
                                   (torch.float32, torch.float16)])
def test_gradients(m, d, yt, ht):
    print("case", m, d, yt, ht, flush=True)
    h = (_rand((m, d), seed=1) * (torch.logspace(-2, 2, m, device="cuda")[:, None] if m > 1 else 1.0)).to(ht)
    w = (1 + _rand((d,), sigma=0.2, seed=3)).to(DTYPES[(m + d) % 3])
    dy, dh = _rand((m, d), yt, 4, 0.1), _rand((m, d), ht, 5, 0.1)
    rstd = ss.fsdp_rms_norm_fp8(h, w, eps=1e-5).rstd
    dx, dw = ss.fsdp_rms_norm_grads(dy, h, w, rstd, dh=dh, dw_dtype=torch.float32)
    assert dx.dtype == ht
    _check_grads(dx, dw, dy, h, w, rstd, dh)
    plain, short = ss.fsdp_rms_norm_grads(dy, h, w, rstd)
    assert short.dtype == w.dtype
    _check_grads(plain, short, dy, h, w, rstd, None)
    one, none = ss.fsdp_rms_norm_grads(dy, h, w, rstd, dh=dh, dw=False)
    assert none is None and torch.equal(_bits(one), _bits(dx))
    none, one = ss.fsdp_rms_norm_grads(dy, h, w, rstd, dx=False, dw_dtype=torch.float32)
    assert none is None and torch.equal(_bits(one), _bits(dw))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,d", [(5, 77), (3, 1601), (4, 2050), (3, 9001)])
def test_gradients_of_strided_rows_and_in_place(m, d, dtype):
    print("case", m, d, dtype, flush=True)
    es = torch.empty(0, dtype=dtype).element_size()
    ld = d + 5
    n = (m - 1) * ld + d
    held = {k: Guarded(n, dtype, offset=3 * es, init=_rand((n,), dtype, i)) for i, k in enumerate(("dy", "h", "dh"))}
    out = Guarded(n, dtype, offset=3 * es)
    rows = {k: torch.as_strided(g.t, (m, d), (ld, 1)) for k, g in {**held, "dx": out}.items()}
    w = _rand((d + 3,), dtype, 9)[3:]
    rstd = ss.fsdp_rms_norm_fp8(rows["h"], w).rstd
    flat = Guarded(d + 5, torch.float32, offset=4)               # dw at its place in a flat gradient
    dx, dw = ss.fsdp_rms_norm_grads(rows["dy"], rows["h"], w, rstd, dh=rows["dh"], dx=rows["dx"], dw=flat.t[5:])
    for k, g in {**held, "dx": out, "dw": flat}.items():
        g.check(k)
    assert (flat.t[:5].view(torch.uint8) == 0xA5).all() and dw.data_ptr() == flat.t[5:].data_ptr()
    gap = torch.as_strided(out.t, (m - 1, 5), (ld, 1), out.t.storage_offset() + d)
    assert (gap.contiguous().view(torch.uint8) == 0xA5).all()
    _check_grads(dx, dw, rows["dy"], rows["h"], w, rstd, rows["dh"])
    want = dx.clone()
    for k in ("dh", "dy"):
        keep = rows[k].clone()
        got, _ = ss.fsdp_rms_norm_grads(rows["dy"], rows["h"], w, rstd, dh=rows["dh"], dx=rows[k], dw=False)
        assert got is rows[k] and torch.equal(_bits(got), _bits(want)), k
        held[k].check(k)
        rows[k].copy_(keep)


def test_no_rows_and_no_features():
    w = torch.ones(40, device="cuda")
    o = ss.fsdp_rms_norm_fp8(torch.empty((0, 40), device="cuda"), w)
    assert o.q.shape == (0, 40) and o.rstd.shape == (0,)
    dx, dw = ss.fsdp_rms_norm_grads(torch.empty((0, 40), device="cuda"), o.h, w, o.rstd)
    assert dx.shape == (0, 40) and torch.equal(dw, torch.zeros(40, device="cuda"))
    assert ss.fsdp_rms_norm_fp8(torch.empty((3, 0), device="cuda"), torch.empty(0, device="cuda")).q.shape == (3, 0)


def test_refusals():
    x, w = _rand((4, 64)), torch.ones(64, device="cuda")
    for f in (lambda: ss.fsdp_rms_norm_fp8(x, w[:63]), lambda: ss.fsdp_rms_norm_fp8(x, w, x[:3]),
              lambda: ss.fsdp_rms_norm_fp8(x, w, h=x), lambda: ss.fsdp_rms_norm_fp8(x.t(), torch.ones(4, device="cuda")),
              lambda: ss.fsdp_rms_norm_fp8(x.clone().requires_grad_(), w),
              lambda: ss.fsdp_rms_norm_fp8(x, w.clone().requires_grad_()),
              lambda: ss.fsdp_rms_norm_fp8(x, w.cpu()), lambda: ss.fsdp_rms_norm_fp8(x, w, x.cpu()),
              lambda: ss.fsdp_rms_norm_fp8(x, w, out=ss.Fp8.empty(4, 65)),
              lambda: ss.fsdp_rms_norm_grads(x, x, w, w[:3]), lambda: ss.fsdp_rms_norm_grads(x, x[:3], w, w[:4])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ss.fsdp_rms_norm_fp8(x.double(), w), lambda: ss.fsdp_rms_norm_grads(x, x, w, w[:4].half()),
              lambda: ss.fsdp_rms_norm_fp8(x, w, x.half(), h=x.clone()),
              lambda: ss.fsdp_rms_norm_grads(x, x, w, w[:4], dh=x.half())):
        with pytest.raises(TypeError):
            f()
    for eps in (-1e-6, math.nan):
        with pytest.raises(ss.FsdpError):
            ss.fsdp_rms_norm_fp8(x, w, eps=eps)
    wide = torch.zeros((2, 32_769), device="cuda")
    with pytest.raises(ss.FsdpError):
        ss.fsdp_rms_norm_fp8(wide, wide[0])
    with torch.no_grad():
        assert ss.fsdp_rms_norm_fp8(x.clone().requires_grad_(), w).q.shape == (4, 64)


def test_gradients_against_differences():
    """Central differences in 64 bits of the formula, at the values that the kernel was given."""
    m, d, eps, step = 3, 40, 1e-3, 1e-5
    x, w, dy, dh = (_rand(s, seed=i) for i, s in enumerate([(m, d), (d,), (m, d), (m, d)]))
    rstd = ss.fsdp_rms_norm_fp8(x, w, eps=eps).rstd
    dx, dw = ss.fsdp_rms_norm_grads(dy, x, w, rstd, dh=dh)
    X, W, DY, DH = (_f64(t) for t in (x, w, dy, dh))

    def loss(X, W):
        r = 1 / np.sqrt((X ** 2).mean(axis=1, keepdims=True) + eps)
        return (X * r * W * DY).sum() + (X * DH).sum()

    for i, j in ((0, 0), (2, 39), (1, 17)):
        e = np.zeros_like(X)
        e[i, j] = step
        diff = (loss(X + e, W) - loss(X - e, W)) / (2 * step)
        assert abs(diff - float(dx[i, j])) < 1e-4, (i, j)
        f = np.zeros_like(W)
        f[j] = step
        diff = (loss(X, W + f) - loss(X, W - f)) / (2 * step)
        assert abs(diff - float(dw[j])) < 1e-4, j


def test_a_units_step_gather_norm_and_product_together():
    """The path: a step, the new shard in 8-bit blocks, the packed all-gather, views of the weights, the norm in
    front of a product, the product, both their gradients into the flat gradient, and the norm of that."""
    world, rank, d, f, m = 2, 1, 128, 384, 40
    shapes = [(d,), (f, d), (128,)]
    P, Pp, S = ss.fsdp_layout([d, f * d, 128], world)
    assert S % 128 == 0
    master = [_rand((S,), seed=q, sigma=0.02) for q in range(world)]
    master[0][:d] += 1                                            # the norm's weight
    unit = dict(master=master[rank], exp_avg=torch.zeros(S, device="cuda"), exp_avg_sq=torch.zeros(S, device="cuda"),
                rank_grads=[_rand((Pp,), torch.bfloat16, 10 + q, 1e-3) for q in range(world)])
    ss.fsdp_step_units([unit], rank, True, ss.AdamWHP(step=1))
    shards = [ss.fsdp_fp8_quantize(t) for t in master]
    packed = ss.fsdp_fp8_gather_packed(shards)
    full = ss.fsdp_fp8_gather(shards, dtype=torch.float32)
    w = ss.fsdp_fp8_views(packed, shapes)[1]
    gamma, plain, _ = ss.fsdp_unflatten_views(full, shapes)
    assert np.array_equal(fp8_ref.values(w.codes.cpu().numpy(), w.scales.cpu().numpy(), d), _f64(plain))
    x, res = _rand((m, d), torch.bfloat16, 20), _rand((m, d), torch.bfloat16, 21)
    o = ss.fsdp_rms_norm_fp8(x, gamma, res, y=torch.empty((m, d), device="cuda"))
    _check_norm(o, x, gamma, res, 1e-6)
    y = ss.fsdp_fp8_linear(o.q, w)
    a, b = fp8_ref.values(o.q.codes.cpu().numpy(), o.q.scales.cpu().numpy(), d), _f64(plain)
    # the product's own tolerance: 7 * 2^-13 of the sum of magnitudes (test_gpu_fp8.py) and half a step of bf16
    assert_within(_f64(y), a @ b.T, (7 * 2.0 ** -13 + d * 2.0 ** -23) * 1.01 * (np.abs(a) @ np.abs(b).T)
                  + 2.0 ** -8 * np.abs(a @ b.T), "y")
    assert torch.equal(y, ss.fsdp_fp8_linear(o.y, w, dtype=torch.bfloat16))
    flat = torch.zeros(Pp, device="cuda")
    views = ss.fsdp_unflatten_views(flat, shapes)
    dn, _ = ss.fsdp_fp8_linear_grads(y, o.y, ss.fsdp_fp8_quantize(plain, form="columns"), dw=views[1])
    dx, _ = ss.fsdp_rms_norm_grads(dn, o.h, gamma, o.rstd, dh=x, dw=views[0])
    _check_grads(dx, views[0], dn, o.h, gamma, o.rstd, x)
    gn = ss.fsdp_grad_norm([flat], 1.0)
    want = math.sqrt(float(flat.double().square().sum()))
    assert want > 0 and abs(float(gn.norm) - want) <= 2.0 ** -23 * want


def test_on_another_stream_and_replayed():
    m, d, n = 300, 1600, 200
    x, res, dy = (_rand((m, d), torch.bfloat16, i) for i in range(3))
    w, lin = torch.ones(d, device="cuda"), ss.fsdp_fp8_quantize(_rand((n, d), seed=4), tile=True)

    def layer(stream=None):
        o = ss.fsdp_rms_norm_fp8(x, w, res, stream=stream)
        y = ss.fsdp_fp8_linear(o.q, lin, stream=stream)
        return (o.h, o.rstd, y, *ss.fsdp_rms_norm_grads(dy, o.h, w, o.rstd, dh=res, stream=stream))

    first = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    others = [layer(side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(a, b) for o in others for a, b in zip(o, first))
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(layer())
    for replay in range(3):
        x.mul_(0.75)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        again = layer()
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, again)), replay
