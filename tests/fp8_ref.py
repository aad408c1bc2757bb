"""8-bit blocks in plain numpy and 64 bits, for the tests: the scale by trying
exponents, each element by a search among all e4m3 magnitudes, ties by the
code's last bit."""
import numpy as np

BLOCK = 128


def _magnitudes():
    c = np.arange(127)                                   # 0x7f is the NaN
    e, m = c >> 3, (c & 7).astype(np.float64)
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e.astype(np.float64) - 7))


GRID = _magnitudes()


def nearest(y):
    """Codes 0..126 of magnitudes y in [0, 448]."""
    hi = np.searchsorted(GRID, y, side="left").clip(0, 126)          # GRID[hi] >= y
    lo = (hi - 1).clip(0, 126)
    up, down = GRID[hi] - y, y - GRID[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0)) | (GRID[hi] == y)
    return np.where(take_hi, hi, lo)


def exponent(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e, of finite amax."""
    e = np.full(amax.shape, -126, dtype=np.int64)
    for _ in range(260):
        more = amax > 448 * np.exp2(e.astype(np.float64))
        if not more.any():
            break
        e += more
    return e


def quantize(x, tile=False):
    """(codes uint8 [rows, nb * 128], scales uint8 [rows or tiles, nb]) of x [rows, cols] (any float dtype)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb, high = -(-cols // BLOCK), BLOCK if tile else 1
    v = np.zeros((-(-rows // high) * high, nb * BLOCK))
    v[:rows, :cols] = x
    v = v.reshape(-1, high, nb, BLOCK)
    amax = np.abs(v).max(axis=(1, 3))                   # NaN if any is
    finite = np.isfinite(amax)
    e = exponent(np.where(finite, amax, 0))
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    f = finite[:, None, :, None]
    y = np.abs(np.where(f, v, 0)) * np.exp2(-e.astype(np.float64))[:, None, :, None]
    code = nearest(y) + 128 * np.signbit(v)
    code = np.where(f, code, 0).astype(np.uint8)
    return code.reshape(-1, nb * BLOCK)[:rows], scales


def values(codes, scales, cols, tile=False):
    """The 64-bit values [rows, cols] that blocks stand for."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    mag = np.append(GRID, np.nan)[codes & 127] * np.where(codes & 128, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    if tile:
        s = np.repeat(s, BLOCK, axis=0)[:codes.shape[0]]
    return (mag * np.repeat(s, BLOCK, axis=1))[:, :cols]
