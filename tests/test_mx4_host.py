"""4-bit microscaled blocks on the host: the tests' own reference against the
format's numbers written out, argument validation of the C entry points (fake,
never-dereferenced pointers) and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import mx4_ref
import sharded_state_amd as ss
from sharded_state_amd import _native as N

FAKE = 1 << 40


def vp(x):
    return ctypes.c_void_p(x)


def test_reference_on_written_out_blocks():
    x = np.zeros((1, 40))
    x[0, :12] = [6, 5, 2.5, 1.75, 0.25, 0.75, 3.5, 7.5, -0.0, -1.25, 0.24, -5.1]
    x[0, 32:35] = [0.001, -0.002, 0.0005]
    codes, scales = mx4_ref.quantize(x)
    # block 0: the largest is 7.5 = 1.875 * 4, e = 0; ties go to the even code
    assert scales.tolist() == [[127, (-9 - 2) + 127]]
    assert mx4_ref.values(codes, scales, 40)[0, :12].tolist() == [6, 4, 2, 2, 0, 1, 4, 6, 0, -1, 0, -6]
    assert codes[0, :6].tolist() == [0x67, 0x44, 0x20, 0x76, 0xa8, 0xf0]
    # block 1: 0.002 = 1.024 * 2^-9
    assert np.array_equal(mx4_ref.values(codes, scales, 40)[0, 32:35], np.array([2, -4, 1]) * 2.0 ** -11)
    assert not codes[0, 18:].any()
    for bad in (np.inf, np.nan):
        x[0, 3] = bad
        c, s = mx4_ref.quantize(x)
        assert s[0, 0] == 255 and not c[0, :16].any() and np.isnan(mx4_ref.values(c, s, 40)[0, :32]).all()
    c, s = mx4_ref.quantize(np.array([[0.0, -0.0], [2.0 ** -149, 2.0 ** -126]]))
    assert s.tolist() == [[0], [0]] and c[0, 0] == 0x80
    assert mx4_ref.values(c, s, 2)[1].tolist() == [0.0, 2.0 ** -126]


def test_quantize_refuses():
    L = N.lib()

    def call(src=FAKE, dt=N.F32, rows=4, cols=64, ld=64, c=FAKE + (1 << 30), s=FAKE + (2 << 30), ct=0, st=0):
        return L.fsdp_mx4_quantize(vp(src), dt, rows, cols, ld, vp(c), vp(s), vp(ct), vp(st), None)

    assert call(dt=4) == N.E_DTYPE
    assert call(rows=-1) == N.E_INVAL and call(cols=-1) == N.E_INVAL
    assert call(ld=63) == N.E_INVAL
    assert call(src=0) == N.E_INVAL
    assert call(c=0) == N.E_INVAL and call(s=0) == N.E_INVAL and call(c=0, s=0) == N.E_INVAL
    assert call(ct=FAKE + (3 << 30)) == N.E_INVAL
    assert call(c=FAKE + (1 << 30) + 8) == N.E_INVAL
    assert call(rows=1 << 40, cols=1 << 40, ld=1 << 40) == N.E_SIZE
    assert call(rows=1 << 40, cols=4, ld=1 << 40) == N.E_SIZE
    assert call(c=FAKE + 1008) == N.E_ALIAS                          # inside src's 1024 bytes
    assert call(s=FAKE + (1 << 30) + 127) == N.E_ALIAS               # the codes' last byte
    assert call(ct=FAKE + (1 << 30), st=FAKE + (3 << 30)) == N.E_ALIAS
    assert call(rows=0) == N.OK and call(cols=0, ld=0, c=0, s=0) == N.OK


def test_gathers_refuse():
    L = N.lib()
    c = [FAKE, FAKE + (1 << 30)]
    s = [FAKE + (2 << 30), FAKE + (3 << 30)]
    out = FAKE + (4 << 30)

    def call(c=c, s=s, world=2, S=64, dt=N.BF16, out=out):
        return L.fsdp_mx4_gather(N.ptr_array(c), N.ptr_array(s), world, S, dt, vp(out), None)

    assert call(world=0) == N.E_INVAL and call(world=129) == N.E_INVAL
    assert call(S=-1) == N.E_INVAL and call(S=1 << 62) == N.E_SIZE
    assert call(dt=9) == N.E_DTYPE and call(out=0) == N.E_INVAL
    assert call(c=[FAKE, 0]) == N.E_INVAL and call(s=[0, s[1]]) == N.E_INVAL
    assert call(c=[FAKE + 8, c[1]]) == N.E_INVAL
    assert call(out=s[1] - 255) == N.E_ALIAS and call(S=0) == N.OK

    def packed(c=c, s=s, S=64, fc=out, fs=FAKE + (5 << 30)):
        return L.fsdp_mx4_gather_packed(N.ptr_array(c), N.ptr_array(s), 2, S, vp(fc), vp(fs), None)

    assert packed(S=65) == N.E_SIZE and "multiple" in L.fsdp_last_error().decode()
    assert packed(fc=0) == N.E_INVAL and packed(fs=0) == N.E_INVAL and packed(fc=out + 4) == N.E_INVAL
    assert packed(c=[0, c[1]]) == N.E_INVAL
    assert packed(c=[out + 32, c[1]]) == N.E_ALIAS                   # shard 0 in the slot of shard 1
    assert packed(fs=out + 63) == N.E_ALIAS
    assert packed(S=0) == N.OK


def test_matmul_refuses():
    L = N.lib()

    def call(a=FAKE, sa=FAKE + (1 << 30), b=FAKE + (2 << 30), sb=FAKE + (3 << 30), m=32, n=64, k=96, dt=N.F32,
             out=FAKE + (4 << 30), ldo=64):
        return L.fsdp_mx4_matmul(vp(a), vp(sa), vp(b), vp(sb), m, n, k, dt, vp(out), ldo, None)

    assert call(dt=3) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(n=-1) == N.E_INVAL and call(k=-1) == N.E_INVAL
    assert call(ldo=63) == N.E_INVAL and call(out=0) == N.E_INVAL
    assert call(a=0) == N.E_INVAL and call(sb=0) == N.E_INVAL
    assert call(a=FAKE + 4) == N.E_INVAL and call(b=FAKE + (2 << 30) + 8) == N.E_INVAL
    assert call(k=(1 << 23) + 1) == N.E_SIZE
    assert call(m=1 << 40, n=1 << 40, ldo=1 << 40) == N.E_SIZE
    assert call(out=FAKE + 32 * 48 - 4) == N.E_ALIAS                 # A's last codes
    assert call(m=0) == N.OK and call(n=0, ldo=0) == N.OK


def test_linear_refuses():
    L = N.lib()
    ws = FAKE + (5 << 30)

    def call(x=FAKE, xdt=N.BF16, m=40, k=96, ldx=96, w=FAKE + (1 << 30), sw=FAKE + (2 << 30), n=64, dt=N.F16,
             out=FAKE + (3 << 30), ldo=64, ws=ws, nbytes=1 << 20):
        return L.fsdp_mx4_linear(vp(x), xdt, m, k, ldx, vp(w), vp(sw), n, dt, vp(out), ldo, vp(ws), nbytes, None)

    assert call(xdt=3) == N.E_DTYPE and call(dt=-1) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(k=-1) == N.E_INVAL and call(n=-1) == N.E_INVAL
    assert call(ldx=95) == N.E_INVAL and call(ldo=63) == N.E_INVAL
    assert call(x=0) == N.E_INVAL and call(w=0) == N.E_INVAL and call(sw=0) == N.E_INVAL and call(out=0) == N.E_INVAL
    assert call(w=FAKE + (1 << 30) + 1) == N.E_INVAL
    assert call(k=(1 << 23) + 1, ldx=1 << 24) == N.E_SIZE
    assert call(out=FAKE + 700) == N.E_ALIAS and call(out=FAKE + (2 << 30) + 190) == N.E_ALIAS
    assert L.fsdp_mx4_linear_workspace(40, 96) == 40 * 3 * 17 + 8
    assert call(nbytes=40 * 3 * 17 + 7) == N.E_SIZE and call(ws=0) == N.E_INVAL and call(ws=ws + 8) == N.E_INVAL
    assert call(ws=FAKE + 1024) == N.E_ALIAS and call(ws=FAKE + (3 << 30) + 16) == N.E_ALIAS
    assert L.fsdp_mx4_linear_workspace(1, 8192) == 0 and L.fsdp_mx4_linear_workspace(0, 8192) == 0
    assert L.fsdp_mx4_linear_workspace(-1, 5) == -1 and L.fsdp_mx4_linear_workspace(1 << 40, 1 << 40) == -1
    assert call(m=0) == N.OK and call(n=0, ldo=0) == N.OK


def test_linear_grads_refuses():
    L = N.lib()
    G = 1 << 30

    def call(dy=FAKE, dydt=N.BF16, lddy=64, x=FAKE + G, xdt=N.BF16, ldx=96, m=40, n=64, k=96, wt=FAKE + 2 * G,
             swt=FAKE + 3 * G, dxdt=N.BF16, dx=FAKE + 4 * G, lddx=96, dwdt=N.F32, dw=FAKE + 5 * G, lddw=96,
             ws=FAKE + 6 * G, nbytes=1 << 20):
        return L.fsdp_mx4_linear_grads(vp(dy), dydt, lddy, vp(x), xdt, ldx, m, n, k, vp(wt), vp(swt), dxdt, vp(dx),
                                       lddx, dwdt, vp(dw), lddw, vp(ws), nbytes, None)

    assert call(dydt=5) == N.E_DTYPE and call(xdt=5) == N.E_DTYPE and call(dxdt=5) == N.E_DTYPE
    assert call(dwdt=5) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(n=-1) == N.E_INVAL and call(k=-1) == N.E_INVAL
    assert call(lddy=63) == N.E_INVAL and call(ldx=95) == N.E_INVAL and call(lddx=95) == N.E_INVAL
    assert call(lddw=95) == N.E_INVAL
    assert call(dy=0) == N.E_INVAL and call(x=0) == N.E_INVAL and call(wt=0) == N.E_INVAL and call(swt=0) == N.E_INVAL
    assert call(wt=FAKE + 2 * G + 8) == N.E_INVAL and call(ws=0) == N.E_INVAL and call(ws=FAKE + 6 * G + 4) == N.E_INVAL
    need = L.fsdp_mx4_linear_grads_workspace(40, 64, 96, 1, 1)
    assert need == (40 * 2 + 64 * 2 + 96 * 2) * 17                       # each a multiple of 16 already
    assert call(nbytes=need - 1) == N.E_SIZE
    assert L.fsdp_mx4_linear_grads_workspace(40, 64, 96, 1, 0) == 40 * 2 * 17
    assert L.fsdp_mx4_linear_grads_workspace(40, -64, 96, 1, 0) == -1
    assert call(dx=FAKE + 64) == N.E_ALIAS and call(dw=FAKE + 4 * G + 64) == N.E_ALIAS
    assert call(ws=FAKE + 5 * G + 1024) == N.E_ALIAS and call(ws=FAKE + 3 * G) == N.E_ALIAS
    assert call(m=1 << 24, lddy=64) == N.E_SIZE                          # dw sums over more than 2^23 tokens
    assert call(dx=0, dw=0, dy=0) == N.OK and call(k=0, ldx=0, lddx=0, lddw=0) == N.OK


def test_binding_refuses():
    z = torch.zeros(4, 64)
    for f in (lambda: ss.fsdp_mx4_quantize(z), lambda: ss.fsdp_mx4_quantize(z, form="diagonal"),
              lambda: ss.fsdp_mx4_gather([])):
        with pytest.raises(ValueError):
            f()
    a = ss.Mx4.empty(4, 70, "cpu")
    assert a.shape == (4, 70) and a.codes.shape == (4, 48) and a.scales.shape == (4, 3)
    with pytest.raises(ValueError):
        ss.Mx4(a.codes, a.scales, 64)                                # two blocks, not three
    with pytest.raises(ValueError):
        ss.Mx4(a.codes[:, :32], a.scales[:, :2], 64)                 # rows not next to each other
    with pytest.raises(ValueError):
        ss.Mx4(a.codes, a.scales[:2], 70)
    with pytest.raises(ValueError):
        ss.fsdp_mx4_matmul(a, a)                                     # on the host
    with pytest.raises(ValueError):
        ss.fsdp_mx4_linear(torch.zeros(2, 64), a)
    with pytest.raises(TypeError):
        ss.fsdp_mx4_linear(torch.zeros(2, 64), z)


def test_views_of_a_packed_unit():
    full = ss.Mx4.empty(1, 32 * 40, "cpu")
    full.scales.copy_(torch.arange(40, dtype=torch.uint8).view(1, 40))
    v = ss.fsdp_mx4_views(full, [(32,), (4, 64), (5,), (3, 32), (27,), (2, 2, 32)])
    assert [x.shape if x is not None else None for x in v] == [(1, 32), (4, 64), None, None, None, (4, 32)]
    assert v[1].scales.tolist() == [[1, 2], [3, 4], [5, 6], [7, 8]]
    # 32 + 256 + 5 + 96 + 27 = 416 elements lie before the last tensor
    assert v[5].codes.data_ptr() == full.codes.data_ptr() + 208 and v[5].scales[0, 0] == 13
    with pytest.raises(ValueError):
        ss.fsdp_mx4_views(full, [(41, 32)])
