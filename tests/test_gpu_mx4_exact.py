"""GPU: products, linear and gradients of 4-bit blocks on whole numbers, where
every partial sum is exact in fp32 and the result is one rounding of the exact
sum: any order, tile or number of waves gives the same values, and a NaN or a
block lost or read twice shows at every length.  And the products of random
blocks within the bound of an fp32 sum, NaN counted as wrong."""
import pytest
import torch

import mx4_ref
import sharded_state_amd as ss
from guards import Guarded
from mx4_check import assert_equal, assert_within, sum_tolerance, whole, whole_product

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
# (rows, rows, sum): few rows, each size of tile, ragged ends of every kind
SHAPES = [(1, 1, 1), (1, 1000, 333), (2, 33, 4096), (5, 70, 32), (16, 512, 1000), (17, 48, 2050), (33, 65, 31),
          (65, 257, 160), (100, 300, 1024), (129, 384, 544), (257, 255, 300), (300, 520, 2080), (7, 1500, 9000),
          (1024, 96, 40), (3000, 5000, 97)]
# tokens up to the ends of what one launch takes (65536 features, 640 blocks) and behind them
LINEAR = [(1, 17, 33), (2, 100, 512), (1, 8200, 700), (3, 16_400, 96), (1, 40, 65_536), (1, 40, 65_568),
          (3, 50, 21_830), (3, 50, 21_857), (16, 31, 1280), (16, 4100, 1281), (17, 300, 1024), (9, 24_600, 97),
          (31, 200, 160), (33, 8197, 96), (2, 40, 32_768), (130, 70, 12_345)]


def _strided(rows, cols, pad, off, dtype, init=None):
    es = torch.empty(0, dtype=dtype).element_size()
    h = Guarded((rows - 1) * (cols + pad) + cols, dtype, offset=off * es)
    t = torch.as_strided(h.t, (rows, cols), (cols + pad, 1))
    if init is not None:
        t.copy_(init)
    return h, t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    x, w = whole((m, k), 1, "cuda"), whole((n, k), 2, "cuda")
    a, b = ss.fsdp_mx4_quantize(x), ss.fsdp_mx4_quantize(w)
    want = whole_product(x, w, dtype)
    for pad, off in ((0, 0), (3, 1)):
        h, y = _strided(m, n, pad, off, dtype)
        ss.fsdp_mx4_matmul(a, b, y)
        h.check("out")
        assert_equal(y, want, "product, rows %d apart" % (n + pad))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_linear(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    x, w = whole((m, k), 3, "cuda"), whole((n, k), 4, "cuda")
    q = ss.fsdp_mx4_quantize(w)
    assert_equal(ss.fsdp_mx4_linear(x.to(dtype), q), whole_product(x, w, dtype), "y")
    hx, xs = _strided(m, k, 5, 1, dtype, x)
    hy, y = _strided(m, n, 1, 1, torch.float32)
    ss.fsdp_mx4_linear(xs, q, y)
    hy.check("y")
    assert_equal(y, whole_product(x, w, torch.float32), "y in fp32, strided")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 40, 70), (17, 1000, 33), (50, 130, 97), (130, 300, 200),
                                   (512, 1100, 1700), (2100, 2110, 2600), (9000, 33, 65)])
def test_gradients(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    dy, x, w = whole((m, n), 5, "cuda"), whole((m, k), 6, "cuda"), whole((n, k), 7, "cuda")
    wt = ss.fsdp_mx4_quantize(w, form="columns")
    dx, dw = ss.fsdp_mx4_linear_grads(dy.to(dtype), x.to(dtype), wt, dw_dtype=torch.float32)
    assert_equal(dx, whole_product(dy, w.T, dtype), "dx")
    assert_equal(dw, whole_product(dy.T, x.T, torch.float32), "dw")
    flat = Guarded(n * k + 5, dtype, offset=dy.to(dtype).element_size())
    ss.fsdp_mx4_linear_grads(dy.to(dtype), x.to(dtype), wt, dx=False, dw=flat.t[5:].view(n, k))
    flat.check("dw")
    assert_equal(flat.t[5:].view(n, k), whole_product(dy.T, x.T, dtype), "dw in the flat gradient")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_of_random_blocks(dtype, m, n, k):
    print("case", dtype, m, n, k, flush=True)
    if m * n > 1 << 20:
        m = 300
    g = torch.Generator(device="cuda")
    g.manual_seed(k)

    def blocks(rows):
        x = torch.randn(rows, k, device="cuda", generator=g) * 2.0 ** torch.randint(-3, 4, (rows, 1), device="cuda",
                                                                                   generator=g)
        q = ss.fsdp_mx4_quantize(x)
        return q, mx4_ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), k)

    (a, va), (b, vb) = blocks(m), blocks(n)
    got = ss.fsdp_mx4_matmul(a, b, dtype=dtype).cpu().double().numpy()
    assert_within(got, va @ vb.T, sum_tolerance(va, vb, dtype), "product")
