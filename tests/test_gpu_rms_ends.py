"""GPU: the norm's codes at both ends of fp32's range.  They are the 64-bit product's,
rounded once: also where that product lies beside a tie between two codes by less than
a fp32 subnormal holds, and where it is larger than fp32's largest.  The reference's
rstd may differ from the kernel's by a few steps of 2^-53, products lie at least 2^-45
of their size away from a tie, so the codes are equal.
"""
import numpy as np
import pytest
import torch

import fp8_ref
import sharded_state_amd as ss

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.detach().cpu().double().numpy()


def _product(h, w, eps):
    H = _f64(h)
    return H * (1 / np.sqrt((H ** 2).sum(axis=1) / H.shape[1] + eps))[:, None] * _f64(w)


def _same(o, z):
    """The blocks of z, which lies far enough from every tie."""
    codes, scales = fp8_ref.quantize(z)
    y = np.abs(z) * np.exp2(127 - np.repeat(scales.astype(np.float64), 128, axis=1)[:, :z.shape[1]])
    y = y[np.isfinite(y)]
    ties = (fp8_ref.GRID[1:] + fp8_ref.GRID[:-1]) / 2
    above = np.searchsorted(ties, y)
    for t in (ties[above.clip(0, len(ties) - 1)], ties[(above - 1).clip(0)]):
        assert (np.abs(y - t) > 2.0 ** -45 * t).all()
    assert np.array_equal(o.q.scales.cpu().numpy(), scales), "scales"
    got = o.q.codes.cpu().numpy()
    bad = got != codes
    assert not bad.any(), "%d codes differ, first at %s: %#x, want %#x" % (bad.sum(), np.argwhere(bad)[0], got[bad][0], codes[bad][0])


@pytest.mark.parametrize("d", [128, 200, 1000, 5000, 9001, 20_001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_codes_beside_ties_of_the_smallest_scales(d, dtype):
    """Weights on the ties between codes of scale bytes 1 to 12 and rows of about 1: products just under and over them."""
    h = torch.ones((4, d), dtype=dtype, device="cuda")
    step = 2.0 ** -23 if dtype is torch.float32 else 2.0 ** -7
    for i, j in ((0, 1), (1, 5), (2, d // 2), (3, d - 1)):
        h[i, j] = 1 + (i + 1) * step
        h[i, ::3] *= -1
    ties = (fp8_ref.GRID[1:] + fp8_ref.GRID[:-1]) / 2
    for s in range(1, 13):
        w = np.resize(ties, d) * 2.0 ** (s - 127)
        w[::128] = 448 * 2.0 ** (s - 127) * 0.9375                   # the block's scale
        w = torch.from_numpy(w).float().cuda()
        o = ss.fsdp_rms_norm_fp8(h, w, eps=0.0)
        _same(o, _product(h, w, 0.0))


@pytest.mark.parametrize("d", [128, 300, 1600, 9001])
def test_codes_of_tiny_and_of_random_products(d):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    h = torch.randn((5, d), device="cuda", generator=g)
    for e in (-149, -140, -134, -130, -126, -120, -112):
        w = torch.randn(d, device="cuda", generator=g) * 2.0 ** e * 16
        _same(ss.fsdp_rms_norm_fp8(h, w, eps=0.0), _product(h, w, 0.0))


@pytest.mark.parametrize("d", [128, 1000, 32_768])
def test_products_over_the_largest_fp32(d):
    """A row of one large element has an rstd that takes it to sqrt(d): times a large weight that is over 2^128, which the
    blocks hold and fp32 does not."""
    h = torch.zeros((4, d), device="cuda")
    h[0, 3], h[1, d - 1], h[2, 64], h[3, 0] = 1.0, -3.0, 7.5, float("inf")
    h[:, 1] += 0.01
    for top in (3.0e38, torch.finfo(torch.float32).max, 1e38):
        w = torch.full((d,), top, device="cuda")
        o = ss.fsdp_rms_norm_fp8(h, w, eps=1e-6, y=True)
        with np.errstate(invalid="ignore"):
            z = _product(h, w, 1e-6)
        _same(o, z)
        assert o.q.scales[0, 0] < 255 and torch.isinf(o.y[0, 3]) and o.q.scales[3, 0] == 255
        back = fp8_ref.values(o.q.codes.cpu().numpy(), o.q.scales.cpu().numpy(), d)
        assert abs(back[0, 3] - z[0, 3]) <= 2.0 ** -4 * z[0, 3]


def test_rstd_of_no_features():
    w = torch.empty(0, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        torch.full((1000,), 5.0, device="cuda")                      # what the allocator would give next
        o = ss.fsdp_rms_norm_fp8(torch.empty((1000, 0), device="cuda"), w, torch.empty((1000, 0), device="cuda"), stream=stream)
        torch.cuda.synchronize()
        assert o.rstd.isnan().all() and o.q.shape == (1000, 0) and o.h.shape == (1000, 0)
        dx, dw = ss.fsdp_rms_norm_grads(o.h, o.h, w, o.rstd)
        assert dx.shape == (1000, 0) and dw.shape == (0,)
