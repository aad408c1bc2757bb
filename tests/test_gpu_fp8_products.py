"""GPU: the 8-bit product where a workgroup makes more than one tile, in the largest
tiles (256 x 256) and in pairs of 128 x 128 a CU, over few and many blocks.  Elements
in {-1, 0, 1, 2} and sums far under 2^24: the fp32 product is exact, and rounded once
to its type.
"""
import pytest
import torch

import sharded_state_amd as ss
from mx4_check import whole

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def _product(x, w, dtype):
    return (x.double() @ w.double().t()).float().to(dtype)


def _same(got, want, what):
    bad = ~(got == want)
    assert not bad.any(), "%s: %d of %d differ, first at %s" % (what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


# 256 x 256: whole tiles, more than a CU takes at once; then with ragged edges.  128 x 128:
# more than 512 tiles, and fewer than 160 of 256 x 256.
@pytest.mark.parametrize("m,n", [(4096, 5120), (4000, 5000), (2816, 3584), (2790, 3500)])
@pytest.mark.parametrize("blocks", [1, 2, 3, 5, 16, 17, 33])
def test_many_tiles_a_workgroup(m, n, blocks):
    k = blocks * 128 - (blocks % 2) * 40
    x, w = whole((m, k), 3 + blocks, "cuda"), whole((n, k), 4 + blocks, "cuda")
    a, b = ss.fsdp_fp8_quantize(x), ss.fsdp_fp8_quantize(w, tile=blocks % 2 == 0)
    for dtype in DTYPES:
        print("case", m, n, k, dtype, flush=True)
        out = torch.full((m, n), float("nan"), dtype=dtype, device="cuda")
        _same(ss.fsdp_fp8_matmul(a, b, out), _product(x, w, dtype), "product")


@pytest.mark.parametrize("m,n,k", [(4096, 5120, 640), (4000, 5000, 2100)])
def test_two_streams_of_the_largest_tiles(m, n, k):
    sets = [(whole((m, k), 20 + i, "cuda"), whole((n, k), 30 + i, "cuda")) for i in range(2)]
    want = [_product(x, w, torch.bfloat16) for x, w in sets]
    ops = [(ss.fsdp_fp8_quantize(x), ss.fsdp_fp8_quantize(w, tile=True)) for x, w in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [[ss.fsdp_fp8_matmul(a, b, stream=s) for _ in range(2)] for (a, b), s in zip(ops, streams)]
        torch.cuda.synchronize()
        for i in range(2):
            for y in got[i]:
                _same(y, want[i], "stream %d" % i)


def test_both_gradients_in_the_largest_tiles():
    """More tiles of each product than CUs, in one launch; whole numbers that blocks hold in either direction."""
    m, n, k = 4096, 4352, 4608
    x, w, dy = whole((m, k), 1, "cuda"), whole((n, k), 2, "cuda"), whole((m, n), 3, "cuda")
    wt = ss.fsdp_fp8_quantize(w, form="columns", tile=True)
    dx, dw = ss.fsdp_fp8_linear_grads(dy, x, wt)
    _same(dx, _product(dy, w.t().contiguous(), torch.float32), "dx")
    _same(dw, _product(dy.t().contiguous(), x.t().contiguous(), torch.float32), "dw")
