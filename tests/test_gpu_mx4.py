"""GPU: 4-bit microscaled blocks -- quantisation, gathers, products, gradients.

Codes, scales and gathered values are exact: they equal the reference's bits.
A product sums K terms in fp32; a sum of K fp32 additions in any order, each off
by at most one step (2^-23 of the running sum, which stays under the sum of
magnitudes), is within K * 2^-23 * sum|a b| of the exact one, and the rounding
to the output's type adds half a step of that type.  Where every partial sum is
a small whole number the product is exact.
"""
import math

import numpy as np
import pytest
import torch

import mx4_ref
import sharded_state_amd as ss
from guards import Guarded

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(shape, dtype=torch.float32, seed=0, sigma=1.0):
    return (torch.randn(shape, device="cuda", generator=_gen(seed)) * sigma).to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _same_blocks(q, x, what):
    codes, scales = mx4_ref.quantize(x)
    torch.cuda.synchronize()
    assert np.array_equal(q.scales.cpu().numpy(), scales), what + ": scales"
    assert np.array_equal(q.codes.cpu().numpy(), codes), what + ": codes"


def _mx4_values(q):
    return mx4_ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.cols)


SHAPES = [(1, 1), (1, 31), (1, 33), (1, 100_003), (3, 32), (5, 77), (64, 64), (33, 257), (256, 96), (130, 1000),
          (1000, 1), (257, 513), (64, 2048)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_rows_and_columns(dtype, shape):
    print("case", dtype, shape, flush=True)
    x = _rand(shape, dtype, seed=shape[1]) * torch.logspace(-3, 3, shape[0], device="cuda").to(dtype)[:, None]
    q = ss.fsdp_mx4_quantize(x)
    t = ss.fsdp_mx4_quantize(x, form="columns")
    b, bt = ss.fsdp_mx4_quantize(x, form="both")
    _same_blocks(q, _f64(x), "rows")
    _same_blocks(t, _f64(x).T, "columns")
    for u, v in ((q, b), (t, bt)):
        assert torch.equal(u.codes, v.codes) and torch.equal(u.scales, v.scales)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_strided_rows_and_any_alignment(dtype):
    es = torch.empty(0, dtype=dtype).element_size()
    for rows, cols, ld, off in ((7, 70, 75, 1), (40, 64, 67, 3), (3, 200, 1001, 5), (1, 333, 333, 7)):
        print("case", dtype, rows, cols, ld, off, flush=True)
        n = (rows - 1) * ld + cols
        h = Guarded(n, dtype, offset=off * es, init=_rand((n,), dtype, seed=cols))
        x = torch.as_strided(h.t, (rows, cols), (ld, 1))
        q, t = ss.fsdp_mx4_quantize(x, form="both")
        _same_blocks(q, _f64(x), "rows")
        _same_blocks(t, _f64(x).T, "columns")
        h.check("src")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quantize_of_every_16_bit_encoding(dtype):
    """Each encoding alone in a block, and each beside a 4.0 (the block's scale then 2^0 up to 7.x)."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    x = bits.view(dtype)
    alone = torch.zeros((1 << 16, 32), dtype=dtype, device="cuda")
    alone[:, 5] = x
    beside = alone.clone()
    beside[:, 9] = 4.0
    for m, what in ((alone, "alone"), (beside, "beside 4"), (alone.flip(0), "flipped")):
        _same_blocks(ss.fsdp_mx4_quantize(m.view(1, -1)), _f64(m).reshape(1, -1), what)


def test_quantize_of_fp32_borders():
    """Around every boundary between codes at many exponents, subnormals, the largest values."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 4.0, 6.0, 0.5], dtype=np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    near = near[:31]
    rows = []
    for e in range(-149, 126):
        r = np.zeros(32, dtype=np.float32)
        with np.errstate(under="ignore"):
            r[:31] = (near.astype(np.float64) * 2.0 ** e).astype(np.float32)
        r[31] = np.float32(4.0 * 2.0 ** e) if 4.0 * 2.0 ** e < 3.4e38 else np.float32(3.4e38)
        rows.append(r)
    rows.append(np.full(32, 3.4028235e38, dtype=np.float32))
    rows.append(np.full(32, -1e-45, dtype=np.float32))
    for bad in (np.inf, -np.inf, np.nan):
        r = np.ones(32, dtype=np.float32)
        r[13] = bad
        rows.append(r)
    x = np.stack(rows)
    _same_blocks(ss.fsdp_mx4_quantize(torch.from_numpy(x).cuda()), x, "rows")
    _same_blocks(ss.fsdp_mx4_quantize(torch.from_numpy(x.T.copy()).cuda(), form="columns"), x, "columns")


def _random_blocks(rows, cols, seed, lo=100, hi=150):
    g = _gen(seed)
    nb = -(-cols // 32)
    codes = torch.randint(0, 256, (rows, nb * 16), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(lo, hi, (rows, nb), dtype=torch.uint8, device="cuda", generator=g)
    return ss.Mx4(codes, scales, cols)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("world,S", [(1, 1), (1, 64), (2, 31), (3, 1000), (4, 8192), (8, 12_345), (128, 40)])
def test_gather_into_the_full_buffer(dtype, world, S):
    print("case", dtype, world, S, flush=True)
    shards = [_random_blocks(1, S, q) for q in range(world)]
    for off in (0, 1):
        h = Guarded(world * S, dtype, offset=off * torch.empty(0, dtype=dtype).element_size())
        assert ss.fsdp_mx4_gather(shards, h.t) is h.t
        h.check("full")
        want = torch.from_numpy(np.concatenate([_mx4_values(s)[0] for s in shards])).to(dtype)
        got = h.t.cpu()
        assert torch.equal(got.view(torch.int32 if got.element_size() == 4 else torch.int16),
                           want.view(torch.int32 if got.element_size() == 4 else torch.int16))


@pytest.mark.parametrize("dtype", DTYPES)
def test_gather_of_every_scale(dtype):
    """All 256 scale bytes and all codes: subnormal, overflowing and NaN values."""
    codes = (torch.arange(256 * 16, device="cuda") % 256).to(torch.uint8).view(1, -1)
    scales = torch.arange(256, device="cuda").to(torch.uint8).view(1, -1)
    got = _f64(ss.fsdp_mx4_gather([ss.Mx4(codes, scales, 256 * 32)], dtype=dtype))
    with np.errstate(over="ignore"):
        want = torch.from_numpy(_mx4_values(ss.Mx4(codes, scales, 256 * 32))[0]).float().to(dtype).double().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    finite = ~np.isnan(want)
    assert np.array_equal(np.signbit(got[finite]), np.signbit(want[finite]))


@pytest.mark.parametrize("world,S", [(1, 32), (2, 96), (8, 4096), (100, 64)])
def test_gather_packed_and_views(world, S):
    print("case", world, S, flush=True)
    full = ss.Mx4.empty(1, world * S)
    full.codes.fill_(0xA5)
    nb = S // 32
    shards = [_random_blocks(1, S, q) for q in range(world)]
    place = world // 2                         # this rank's shard already in its slot
    full.codes[:, place * nb * 16:(place + 1) * nb * 16] = shards[place].codes
    full.scales[:, place * nb:(place + 1) * nb] = shards[place].scales
    if (place * nb * 16) % 16 == 0:
        shards[place] = ss.Mx4(full.codes[:, place * nb * 16:(place + 1) * nb * 16],
                               full.scales[:, place * nb:(place + 1) * nb], S)
    want_c, want_s = torch.cat([s.codes for s in shards], 1), torch.cat([s.scales for s in shards], 1)
    assert ss.fsdp_mx4_gather_packed(shards, full) is full
    assert torch.equal(full.codes, want_c) and torch.equal(full.scales, want_s)
    w = ss.fsdp_mx4_views(full, [(world * S // 32, 32)])[0]
    assert np.array_equal(_mx4_values(w).reshape(-1), _mx4_values(full)[0])


PRODUCTS = [(1, 1, 1), (1, 64, 64), (1, 1000, 333), (2, 33, 4096), (5, 70, 32), (16, 512, 1000), (17, 48, 2050),
            (31, 100, 96), (32, 32, 64), (33, 65, 31), (64, 200, 512), (65, 257, 160), (100, 300, 1024),
            (128, 128, 256), (129, 384, 544), (256, 256, 512), (257, 255, 300), (300, 520, 2080), (7, 1500, 9000),
            (512, 640, 8192), (1024, 96, 40)]


def _check_product(got, va, vb, dtype, what):
    want = va @ vb.T
    room = np.abs(va) @ np.abs(vb).T
    k = va.shape[1]
    half = torch.finfo(dtype).eps / 2
    tol = k * 2.0 ** -23 * room * (1 + half) + half * np.abs(want) + torch.finfo(dtype).smallest_normal * half
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d off, first at %s: %r, want %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    a, b = _random_blocks(m, k, 1, 115, 125), _random_blocks(n, k, 2, 115, 125)
    va, vb = _mx4_values(a), _mx4_values(b)
    if k % 32:                                  # the format's zeros behind the last column
        for q in (a, b):
            v = q.codes.view(q.rows, -1, 16)
            tail = k % 32
            v[:, -1, (tail + 1) // 2:] = 0
            if tail % 2:
                v[:, -1, tail // 2] &= 15
    out = Guarded(m * n, dtype)
    assert ss.fsdp_mx4_matmul(a, b, out.t.view(m, n)).shape == (m, n)
    out.check("out")
    _check_product(_f64(out.t).reshape(m, n), va, vb, dtype, "product")


@pytest.mark.parametrize("m,n,k", [(1, 700, 4096), (16, 96, 8192), (40, 64, 2048), (130, 260, 1000), (300, 300, 5000),
                                   (512, 512, 4096)])
def test_product_of_whole_numbers_is_exact(m, n, k):
    """Elements in {-1, 0, 1, 2}, sums far under 2^24: the fp32 product is exact."""
    x = torch.randint(-1, 3, (m, k), device="cuda", generator=_gen(3)).float()
    w = torch.randint(-1, 3, (n, k), device="cuda", generator=_gen(4)).float()
    got = ss.fsdp_mx4_matmul(ss.fsdp_mx4_quantize(x), ss.fsdp_mx4_quantize(w), dtype=torch.float32)
    want = _f64(x) @ _f64(w).T
    assert np.array_equal(_f64(got), want)


@pytest.mark.parametrize("m,n,k", [(3, 50, 96), (20, 70, 160), (100, 300, 96), (300, 600, 128)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_product_into_strided_rows_at_any_alignment(m, n, k, dtype):
    es = torch.empty(0, dtype=dtype).element_size()
    a, b = _random_blocks(m, k, 5, 120, 125), _random_blocks(n, k, 6, 120, 125)
    for pad, off in ((0, 1), (3, 0), (8, 5)):
        ldo = n + pad
        h = Guarded((m - 1) * ldo + n, dtype, offset=off * es)
        before = h.t.clone()
        ss.fsdp_mx4_matmul(a, b, torch.as_strided(h.t, (m, n), (ldo, 1)))
        h.check("out")
        got = torch.as_strided(h.t, (m, n), (ldo, 1))
        _check_product(_f64(got), _mx4_values(a), _mx4_values(b), dtype, "strided")
        if pad and m > 1:                        # what lies between the rows is left as it was
            gap = torch.as_strided(h.t, (m - 1, pad), (ldo, 1), h.t.storage_offset() + n)
            was = torch.as_strided(before, (m - 1, pad), (ldo, 1), n)
            i = torch.int32 if es == 4 else torch.int16
            assert torch.equal(gap.contiguous().view(i), was.contiguous().view(i))


@pytest.mark.parametrize("m,n,k", [(2, 40, 128), (20, 70, 160), (70, 64, 288), (300, 270, 320)])
def test_product_with_nan_blocks_and_extreme_scales(m, n, k):
    a, b = _random_blocks(m, k, 7, 120, 125), _random_blocks(n, k, 8, 120, 125)
    a.scales[m - 1, k // 32 - 1] = 255           # the last row's last block
    b.scales[3, 0] = 255
    got = _f64(ss.fsdp_mx4_matmul(a, b, dtype=torch.float32))
    va, vb = _mx4_values(a), _mx4_values(b)
    nan = np.zeros((m, n), dtype=bool)
    nan[m - 1], nan[:, 3] = True, True
    assert np.array_equal(np.isnan(got), nan)
    ok_r, ok_c = [r for r in range(m) if r != m - 1], [c for c in range(n) if c != 3]
    _check_product(got[np.ix_(ok_r, ok_c)], va[ok_r], vb[ok_c], torch.float32, "beside NaN")
    # 2^-127 * 2^127 scales: exact
    a, b = _random_blocks(m, k, 9), _random_blocks(n, k, 10)
    a.scales.fill_(0)
    b.scales.fill_(254)
    got = _f64(ss.fsdp_mx4_matmul(a, b, dtype=torch.float32))
    assert np.array_equal(got, _mx4_values(a) @ _mx4_values(b).T)


@pytest.mark.parametrize("m,n,k", [(2, 40, 128), (20, 70, 160), (70, 64, 288), (200, 270, 320), (3000, 5000, 96)])
def test_product_of_zeros_with_the_largest_scales(m, n, k):
    """Zero codes (of both signs) give zeros whatever the scales; what overflows fp32 is infinite."""
    a, b = _random_blocks(m, k, 11, 254, 255), _random_blocks(n, k, 12, 254, 255)
    a.codes[::2] &= 0x88                         # zeros
    b.codes.fill_(0x22)                          # ones
    a.codes[1::2] = 0x22
    got = ss.fsdp_mx4_matmul(a, b, dtype=torch.float32)
    assert (got[::2] == 0).all()
    assert (got[1::2] == float("inf")).all()


def test_product_of_empty_operands():
    a, b = ss.Mx4.empty(3, 0), ss.Mx4.empty(5, 0)
    assert torch.equal(ss.fsdp_mx4_matmul(a, b, dtype=torch.float32), torch.zeros(3, 5, device="cuda"))
    a, b = ss.Mx4.empty(0, 64), ss.Mx4.empty(5, 64)
    assert ss.fsdp_mx4_matmul(a, b).shape == (0, 5)
    assert ss.fsdp_mx4_quantize(torch.empty(0, device="cuda")).shape == (1, 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(1, 96, 200), (50, 130, 97), (300, 260, 290)])
def test_linear_and_its_gradients_against_the_formula(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    x, w, dy = _rand((m, k), dtype, 1), _rand((n, k), dtype, 2, 0.05), _rand((m, n), dtype, 3, 0.01)

    def q(t):
        return mx4_ref.values(*mx4_ref.quantize(t), t.shape[1])

    X, W, DY = _f64(x), _f64(w), _f64(dy)
    y = ss.fsdp_mx4_linear(x, ss.fsdp_mx4_quantize(w))
    _check_product(_f64(y), q(X), q(W), dtype, "y")
    flat = Guarded(n * k + 5, torch.float32, offset=4)          # dw at its place in a flat gradient
    dx, dw = ss.fsdp_mx4_linear_grads(dy, x, ss.fsdp_mx4_quantize(w, form="columns"), dw=flat.t[5:].view(n, k))
    flat.check("dw")
    assert dx.dtype == dtype and dw.data_ptr() == flat.t[5:].data_ptr()
    _check_product(_f64(dx), q(DY), q(W.T), dtype, "dx")
    _check_product(_f64(dw), q(DY.T), q(X.T), torch.float32, "dw")
    wt = ss.fsdp_mx4_quantize(w, form="columns")
    alone, none = ss.fsdp_mx4_linear_grads(dy, x, wt, dw=False)
    assert none is None and torch.equal(alone, dx)
    none, alone = ss.fsdp_mx4_linear_grads(dy, x, wt, dx=False, dw_dtype=torch.float32)
    assert none is None and torch.equal(alone, dw)


@pytest.mark.parametrize("m,n,k", [(3, 40, 70), (17, 1000, 33), (130, 300, 200), (300, 1100, 140), (512, 1100, 1700),
                                   (2100, 2110, 2600)])
def test_gradients_together_and_alone(m, n, k):
    """Both products in a launch give what each gives alone, and dy and x of one
    dtype, quantised in one launch, what they give in two dtypes: each element's sum
    runs in one order whatever the tiles."""
    print("case", m, n, k, flush=True)
    x, w = _rand((m, k), torch.bfloat16, 1), _rand((n, k), torch.bfloat16, 2, 0.05)
    dy = _rand((m, n), torch.bfloat16, 3, 0.01)
    wt = ss.fsdp_mx4_quantize(w, form="columns")
    same = ss.fsdp_mx4_linear_grads(dy, x, wt)
    for out in (torch.float16, torch.float32):
        alone = ss.fsdp_mx4_linear_grads(dy, x, wt, dx=False, dw_dtype=out)[1]
        together = ss.fsdp_mx4_linear_grads(dy, x, wt, dw_dtype=out)[1]
        assert together.dtype == out and torch.equal(alone, together)
    assert torch.equal(ss.fsdp_mx4_linear_grads(dy, x, wt, dw=False)[0], same[0])
    for a, b in ((dy.float(), x), (dy, x.float()), (dy.float(), x.float())):
        dx, dw = ss.fsdp_mx4_linear_grads(a, b, wt)
        assert torch.equal(dx.to(torch.bfloat16), same[0]) and torch.equal(dw.to(torch.bfloat16), same[1])


def test_gradients_of_no_tokens():
    x, dy = torch.empty(0, 64, device="cuda"), torch.empty(0, 96, device="cuda")
    wt = ss.fsdp_mx4_quantize(_rand((96, 64)), form="columns")
    dx, dw = ss.fsdp_mx4_linear_grads(dy, x, wt)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(96, 64, device="cuda"))
    assert ss.fsdp_mx4_linear(x, ss.fsdp_mx4_quantize(_rand((96, 64)))).shape == (0, 96)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 17, 33), (2, 100, 512), (1, 8200, 700), (3, 16400, 96),
                                   (16, 1280, 5000), (17, 300, 1024), (31, 8192 + 5, 160), (32, 16384 + 48, 544),
                                   (33, 200, 96), (5, 1600, 4097), (32, 65, 9000), (1, 40, 65_536), (1, 40, 65_568),
                                   (3, 50, 21_830), (3, 50, 21_857), (2, 33, 2050), (16, 31, 1280), (16, 4100, 1281),
                                   (9, 24_600, 97), (1, 15, 16_000)])
def test_linear_of_few_tokens(dtype, m, n, k):
    """Few tokens in one launch, and more: strided and unaligned x and y, and the
    same values as quantisation and product one after the other."""
    print("case", dtype, m, n, k, flush=True)
    es = torch.empty(0, dtype=dtype).element_size()
    w = _random_blocks(n, k, 3, 110, 120)
    for pad, off in ((0, 0), (3, 1)):
        hx = Guarded((m - 1) * (k + pad) + k, dtype, offset=off * es, init=_rand(((m - 1) * (k + pad) + k,), dtype, k))
        x = torch.as_strided(hx.t, (m, k), (k + pad, 1))
        hy = Guarded((m - 1) * (n + pad) + n, dtype, offset=off * es)
        y = torch.as_strided(hy.t, (m, n), (n + pad, 1))
        assert ss.fsdp_mx4_linear(x, w, y) is y
        hy.check("y")
        q = ss.fsdp_mx4_quantize(x)
        _check_product(_f64(y), _mx4_values(q), _mx4_values(w), dtype, "y")
        if pad and m > 1:
            gap = torch.as_strided(hy.t, (m - 1, pad), (n + pad, 1), hy.t.storage_offset() + n)
            assert (gap.contiguous().view(torch.uint8) == 0xA5).all()
    assert ss.fsdp_mx4_linear(x, w).dtype == dtype
    assert torch.equal(ss.fsdp_mx4_linear(x, w), ss.fsdp_mx4_linear(x, w))


def test_linear_of_few_tokens_with_values_that_are_not_finite():
    m, n, k = 4, 40, 300
    x, w = _rand((m, k), torch.bfloat16, 1), _random_blocks(n, k, 2, 110, 120)
    x[1, 299], x[2, 0] = math.nan, math.inf
    w.scales[7, 3] = 255
    y = ss.fsdp_mx4_linear(x, w)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[1], nan[2], nan[:, 7] = True, True, True
    assert torch.equal(torch.isnan(y), nan)
    assert torch.equal(y.isnan(), ss.fsdp_mx4_matmul(ss.fsdp_mx4_quantize(x), w).isnan())


def test_gradients_against_differences():
    """Whole numbers that blocks hold exactly in either direction: y is bilinear
    there, so moving one element from one of them to another changes
    sum(y * dy) by exactly the gradient times the move."""
    m, n, k = 45, 70, 52
    pick = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], device="cuda").float()

    def whole(shape, seed):
        return pick[torch.randint(0, 11, shape, device="cuda", generator=_gen(seed))]

    x, w, dy = whole((m, k), 1), whole((n, k), 2), whole((m, n), 3)

    def loss(x, w):
        y = ss.fsdp_mx4_linear(x, ss.fsdp_mx4_quantize(w))
        return float((y.double() * dy.double()).sum())

    dx, dw = ss.fsdp_mx4_linear_grads(dy, x, ss.fsdp_mx4_quantize(w, form="columns"))
    base = loss(x, w)
    for i, j in ((0, 0), (44, 51), (17, 33), (31, 32)):
        for t, g in ((x, dx), (w, dw)):
            move = t.clone()
            move[i, j] = 2.0 if float(t[i, j]) != 2.0 else -1.0
            h = float(move[i, j] - t[i, j])
            change = (loss(move, w) if t is x else loss(x, move)) - base
            assert change == h * float(g[i, j]), (i, j, change, h, float(g[i, j]))


def test_a_units_step_gather_and_product_together():
    """The path: norm, clipped step, the new shard in 4-bit blocks, the packed
    all-gather, a view of a weight, and a product with it; then its gradients
    into the flat gradient, and the norm of that."""
    world, rank, d, f = 2, 1, 64, 96
    shapes = [(f, d), (d, f), (64,)]
    numels = [f * d, d * f, 64]
    P, Pp, S = ss.fsdp_layout(numels, world)
    assert S % 32 == 0
    master = [_rand((S,), seed=q, sigma=0.02) for q in range(world)]
    grads = [_rand((Pp,), torch.bfloat16, 10 + q, 1e-3) for q in range(world)]
    zeros = [torch.zeros(S, device="cuda") for _ in range(2)]
    unit = dict(master=master[rank], exp_avg=zeros[0], exp_avg_sq=zeros[1], rank_grads=grads)
    gn = ss.fsdp_grad_norm_units([unit], rank, True, 0.05)
    ss.fsdp_step_units([unit], rank, True, ss.AdamWHP(step=1), clip=gn)
    packed = ss.fsdp_mx4_gather_packed([ss.fsdp_mx4_quantize(m) for m in master])
    full = ss.fsdp_mx4_gather([ss.fsdp_mx4_quantize(m) for m in master], dtype=torch.float32)
    assert np.array_equal(_mx4_values(packed)[0], _f64(full))
    w = ss.fsdp_mx4_views(packed, shapes)[0]
    plain = ss.fsdp_unflatten_views(full, shapes)[0]
    assert np.array_equal(_mx4_values(w), _f64(plain))
    x = _rand((40, d), torch.bfloat16, 20)
    y = ss.fsdp_mx4_linear(x, w)
    xq = mx4_ref.values(*mx4_ref.quantize(_f64(x)), d)
    _check_product(_f64(y), xq, _f64(plain), torch.bfloat16, "y")
    flat = torch.zeros(Pp, device="cuda")
    views = ss.fsdp_unflatten_views(flat, shapes)
    ss.fsdp_mx4_linear_grads(y, x, ss.fsdp_mx4_quantize(plain, form="columns"), dw=views[0])
    gn = ss.fsdp_grad_norm([flat], 1.0)
    want = math.sqrt(float(flat.double().square().sum()))
    assert want > 0 and abs(float(gn.norm) - want) <= 2.0 ** -23 * want


def test_on_another_stream_and_replayed():
    m, n, k = 200, 300, 256
    w = ss.fsdp_mx4_quantize(_rand((n, k), torch.bfloat16, 1))
    wt = ss.fsdp_mx4_quantize(_rand((n, k), torch.bfloat16, 1), form="columns")
    x, dy = _rand((m, k), torch.bfloat16, 2), _rand((m, n), torch.bfloat16, 3)
    y0 = ss.fsdp_mx4_linear(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys = [ss.fsdp_mx4_linear(x, w, stream=side) for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(y0, y) for y in ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ss.fsdp_mx4_linear(x, w)
        dx, dw = ss.fsdp_mx4_linear_grads(dy, x, wt)
    for replay in range(3):
        x.mul_(0.75)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        y1 = ss.fsdp_mx4_linear(x, w)
        dx1, dw1 = ss.fsdp_mx4_linear_grads(dy, x, wt)
        torch.cuda.synchronize()
        assert torch.equal(y, y1) and torch.equal(dx, dx1) and torch.equal(dw, dw1), replay
