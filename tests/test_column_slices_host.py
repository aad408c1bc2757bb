"""Column slices of one buffer as operands and results of the 4-bit calls: taken
where they are apart, refused where they overlap (the host's checks, addresses that
nothing dereferences)."""
import ctypes

import pytest
import torch

from sharded_state_amd import _native as N

FAKE = 1 << 40
G = 1 << 30


def vp(x):
    return ctypes.c_void_p(x)


def _linear(x, ldx, out, ldo, m=40, k=96, n=64, xdt=N.BF16, dt=N.BF16):
    return N.lib().fsdp_mx4_linear(vp(x), xdt, m, k, ldx, vp(FAKE + G), vp(FAKE + 2 * G), n, dt, vp(out), ldo,
                                   vp(FAKE + 3 * G), 1 << 20, None)


def _grads(dy, lddy, x, ldx, dx, lddx, dw, lddw, m=40, n=64, k=96):
    return N.lib().fsdp_mx4_linear_grads(vp(dy), N.BF16, lddy, vp(x), N.BF16, ldx, m, n, k, vp(FAKE + 2 * G),
                                         vp(FAKE + 3 * G), N.BF16, vp(dx), lddx, N.BF16, vp(dw), lddw,
                                         vp(FAKE + 4 * G), 1 << 20, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses lie nowhere: only the host's checks run")
@pytest.mark.parametrize("m", [3, 40])
def test_column_slices_of_one_buffer_do_not_overlap(m):
    ld = 96 + 64                                     # x, then out, in rows of 160
    assert _linear(FAKE, ld, FAKE + 2 * 96, ld, m=m) == N.E_HIP
    assert _linear(FAKE + 2 * 64, ld, FAKE, ld, m=m) == N.E_HIP          # out first
    assert _linear(FAKE, 200, FAKE + 2 * 100, 200, m=m) == N.E_HIP       # room before, between and behind
    assert _linear(FAKE, ld, FAKE + 2 * (96 + 7 * ld), ld, m=m) == N.E_HIP    # out some rows further down
    # dy, x, dx, dw in rows of 64 + 3 * 96
    assert _grads(FAKE, 352, FAKE + 2 * 64, 352, FAKE + 2 * 160, 352, FAKE + 2 * 256, 352, m=m) == N.E_HIP
    one = _linear(FAKE, ld, FAKE + 2 * (ld + 96), 64, m=1)               # a single row
    assert one == N.E_HIP


@pytest.mark.parametrize("m", [3, 40])
def test_column_slices_that_overlap_are_refused(m):
    ld = 96 + 64
    assert _linear(FAKE, ld, FAKE + 2 * 95, ld, m=m) == N.E_ALIAS        # x's last column
    assert _linear(FAKE, ld, FAKE + 2 * 97, ld, m=m) == N.E_ALIAS        # the next row's first
    assert _linear(FAKE, ld, FAKE + 2 * 96, ld + 1, m=m) == N.E_ALIAS    # rows drift into each other
    assert _linear(FAKE, ld, FAKE + 2 * 95 + 1, ld, m=m) == N.E_ALIAS    # half an element
    assert _linear(FAKE, ld, FAKE + 2 * 96, ld, m=m, dt=N.F32) == N.E_ALIAS      # rows of other bytes
    assert _linear(FAKE + 2 * 64, ld, FAKE + 2, ld, m=m) == N.E_ALIAS
    assert _grads(FAKE, 352, FAKE + 2 * 64, 352, FAKE + 2 * 160, 352, FAKE + 2 * 255, 352, m=m) == N.E_ALIAS
    assert _grads(FAKE, 352, FAKE + 2 * 64, 352, FAKE + 2 * 159, 352, FAKE + 2 * 256, 352, m=m) == N.E_ALIAS
