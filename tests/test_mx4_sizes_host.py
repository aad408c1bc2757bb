"""Sizes that the 4-bit calls refuse by name before anything is launched (fake,
never-dereferenced addresses)."""
import ctypes

from sharded_state_amd import _native as N

FAKE = 1 << 40


def vp(x):
    return ctypes.c_void_p(x)


def test_more_column_tiles_than_are_counted():
    L = N.lib()
    for rows, cols in ((1 << 40, 1), (1, 1 << 40), ((1 << 38) + 1, 1)):
        assert L.fsdp_mx4_quantize(vp(FAKE), N.BF16, rows, cols, cols, None, None, vp(1 << 50), vp(1 << 54),
                                   None) == N.E_SIZE
        assert "tiles" in L.fsdp_last_error().decode()
    rc = L.fsdp_mx4_linear_grads(vp(FAKE), N.BF16, 1 << 40, vp(FAKE - 4096), N.BF16, 2, 1, 1 << 40, 2, None, None, N.BF16,
                                 None, 0, N.BF16, vp(1 << 50), 2, vp(1 << 52), 1 << 50, None)
    assert rc == N.E_SIZE and "tiles" in L.fsdp_last_error().decode()
