"""Comparisons of the 4-bit products' results that nothing slips through: a NaN
fails like any other wrong value, and sums of whole numbers are compared exactly,
so that one lost or doubled block shows at any length of the sum."""
import numpy as np
import torch


def assert_within(got, want, tol, what):
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= tol)          # a NaN is not within anything
    assert not bad.any(), "%s: %d of %d off, first at %s: %r, want %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])


def sum_tolerance(va, vb, dtype):
    """Bound of a sum of k fp32 products in any order, each addition off by at most
    one step (2^-23) of what stays under the sum of magnitudes, then rounded to
    dtype (half a step of it, or of its subnormals)."""
    want, room = va @ vb.T, np.abs(va) @ np.abs(vb).T
    half = torch.finfo(dtype).eps / 2
    return (va.shape[1] * 2.0 ** -23 * room * (1 + half) + half * np.abs(want)
            + torch.finfo(dtype).smallest_normal * half)


def whole(shape, seed, device="cpu"):
    """Whole numbers from -1 to 2: a 4-bit block holds each of them exactly whatever
    the others are, and the products' sums stay under 2^24, exact in fp32."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randint(-1, 3, shape, device=device, generator=g).float()


def whole_product(x, w, dtype):
    """x w^T of whole numbers, rounded once to dtype."""
    s = x.cpu().double() @ w.cpu().double().T
    assert s.numel() == 0 or float(s.abs().max()) < 2 ** 24
    return s.float().to(dtype)


def assert_equal(got, want, what):
    got = got.detach().cpu()
    assert got.shape == want.shape and got.dtype == want.dtype, (what, got.shape, got.dtype)
    bad = ~(got == want)
    assert not bad.any(), "%s: %d of %d differ, first at %s: %r, want %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]))
