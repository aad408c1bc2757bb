"""GPU: the 8-bit products at their limits and at the borders between their kernels:
the longest sum, the most blocks that few tokens' kernel holds scales of, the sizes
where a linear product begins to quantise apart.  Elements in {-1, 0, 1, 2}, sums
under 2^24: exact.
"""
import pytest
import torch

import sharded_state_amd as ss

pytestmark = pytest.mark.gpu

CODES = (0x00, 0x38, 0xb8, 0x40)                                 # 0, 1, -1, 2
VALUES = (0.0, 1.0, -1.0, 2.0)
MAX_K = 1 << 22


def _blocks(rows, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = ss.Fp8.empty(rows, cols)
    table = torch.tensor(CODES, dtype=torch.uint8, device="cuda")
    for i in range(0, rows, 256):                                # the table's index takes eight bytes an element
        part = q.codes[i:i + 256]
        part.copy_(table[torch.randint(0, 4, part.shape, device="cuda", generator=g)])
    q.codes[:, cols:] = 0
    q.scales.fill_(127)
    return q


def _values(codes):
    table = torch.zeros(256, device="cuda")
    table[list(CODES)] = torch.tensor(VALUES, device="cuda")
    return table[codes.int()]


def _product(a, b):
    want = torch.zeros((a.rows, b.rows), dtype=torch.float64, device="cuda")
    for k in range(0, a.codes.shape[1], 1 << 16):                # a part's sums stay under 2^24: exact in fp32
        want += _values(a.codes[:, k:k + (1 << 16)]) @ _values(b.codes[:, k:k + (1 << 16)]).t().contiguous()
    assert float(want.abs().max()) < 2 ** 24
    return want.float()


def _same(got, want):
    bad = ~(got == want)
    assert not bad.any(), "%d of %d differ, first at %s" % (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("m,n,k", [(3, 5, MAX_K), (70, 40, MAX_K - 129), (300, 520, MAX_K), (2560, 4096, MAX_K),
                                   (16, 40, 2048 * 128), (16, 40, 2048 * 128 + 1), (1, 4200, 2048 * 128), (16, 4200, 2048 * 128),
                                   (7, 4200, 2047 * 128 - 5), (16, 4200, 2049 * 128), (16, 24_576, 300), (16, 24_592, 300),
                                   (17, 24_592, 300)])
def test_product(m, n, k):
    print("case", m, n, k, flush=True)
    a, b = _blocks(m, k, 1), _blocks(n, k, 2)
    _same(ss.fsdp_fp8_matmul(a, b, dtype=torch.float32), _product(a, b))


@pytest.mark.parametrize("m,n,k", [(1, 40, 32_768), (1, 40, 32_769), (4, 40, 8192), (4, 40, 8193), (3, 40, 85 * 128),
                                   (5, 40, 12 * 128), (5, 40, 13 * 128), (16, 40, 512), (16, 40, 513), (17, 40, 128), (17, 40, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_linear(m, n, k, dtype):
    print("case", m, n, k, dtype, flush=True)
    x, w = _blocks(m, k, 3), _blocks(n, k, 4)
    given = _values(x.codes)[:, :k].to(dtype)
    got = ss.fsdp_fp8_linear(given, w, dtype=torch.float32)
    _same(got, _product(x, w))
    assert torch.equal(got, ss.fsdp_fp8_linear(given, w, dtype=torch.float32))


def test_a_longer_sum_is_refused():
    a, b = ss.Fp8.empty(2, MAX_K + 1), ss.Fp8.empty(3, MAX_K + 1)
    with pytest.raises(ss.FsdpError):
        ss.fsdp_fp8_matmul(a, b)
    with pytest.raises(ss.FsdpError):
        ss.fsdp_fp8_linear(torch.zeros(2, MAX_K + 1, device="cuda"), b)
