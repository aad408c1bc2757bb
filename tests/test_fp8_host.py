"""8-bit blocks and the norm in front of them on the host: the tests' own
reference against the format's numbers written out, argument validation of the C
entry points (fake, never-dereferenced pointers) and of the binding."""
import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch

import fp8_ref
import sharded_state_amd as ss
from sharded_state_amd import _native as N

FAKE = 1 << 40
G = 1 << 30


def vp(x):
    return ctypes.c_void_p(x)


def test_reference_on_written_out_blocks():
    x = np.zeros((1, 200))
    # the largest is 448 * 2^-2: e = -2; steps of 32 in the top binade, of 2^-9 at the bottom
    x[0, :8] = np.array([448, 432, 400, -17, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -0.0]) / 4
    x[0, 128:131] = [1.0, 0.9375, -0.97]
    codes, scales = fp8_ref.quantize(x)
    assert scales.tolist() == [[125, 119]]                            # 1 = 256 * 2^-8
    got = fp8_ref.values(codes, scales, 200)[0]
    assert (got[:8] * 4).tolist() == [448, 448, 384, -16, 2.0 ** -9, 0, 2 * 2.0 ** -9, 0]   # ties to the even code
    assert got[128:131].tolist() == [1.0, 0.9375, -1.0]
    assert codes[0, :8].tolist() == [0x7e, 0x7e, 0x7c, 0xd8, 1, 0, 2, 0x80] and not codes[0, 131:].any()
    # just over 448 * 2^e the next exponent is taken: nothing saturates
    c, s = fp8_ref.quantize(np.array([[448.0], [np.nextafter(np.float32(448), np.float32(449))]]))
    assert s.tolist() == [[127], [128]] and c[0, 0] == 0x7e
    for bad in (np.inf, np.nan):
        x[0, 3] = bad
        c, s = fp8_ref.quantize(x)
        assert s[0, 0] == 255 and not c[0, :128].any() and np.isnan(fp8_ref.values(c, s, 200)[0, :128]).all()
    c, s = fp8_ref.quantize(np.array([[0.0, -0.0], [2.0 ** -149, 448 * 2.0 ** -126]]))
    assert s.tolist() == [[1], [1]] and c[:, :2].tolist() == [[0, 0x80], [0, 0x7e]]
    t = np.ones((130, 3))
    t[129, 2] = 1000
    c, s = fp8_ref.quantize(t, tile=True)
    assert s.tolist() == [[119], [129]] and fp8_ref.values(c, s, 3, tile=True)[128, 0] == 1.0


def test_reference_is_torchs_rounding():
    x = np.random.default_rng(0).normal(size=5000).astype(np.float32) * 100
    x = x[np.abs(x) < 448]
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8_ref.nearest(np.abs(x.astype(np.float64))), t & 127)


def test_quantize_refuses():
    L = N.lib()

    def call(src=FAKE, dt=N.F32, rows=4, cols=256, ld=256, tile=0, c=FAKE + G, s=FAKE + 2 * G, ct=0, st=0):
        return L.fsdp_fp8_quantize(vp(src), dt, rows, cols, ld, tile, vp(c), vp(s), vp(ct), vp(st), None)

    assert call(dt=4) == N.E_DTYPE
    assert call(rows=-1) == N.E_INVAL and call(cols=-1) == N.E_INVAL
    assert call(ld=255) == N.E_INVAL
    assert call(src=0) == N.E_INVAL
    assert call(c=0) == N.E_INVAL and call(s=0) == N.E_INVAL and call(c=0, s=0) == N.E_INVAL
    assert call(ct=FAKE + 3 * G) == N.E_INVAL
    assert call(c=FAKE + G + 8) == N.E_INVAL and call(ct=FAKE + 3 * G + 8, st=FAKE + 4 * G) == N.E_INVAL
    assert call(rows=1 << 40, cols=1 << 40, ld=1 << 40) == N.E_SIZE
    assert call(rows=1 << 40, cols=4, ld=1 << 40) == N.E_SIZE
    assert call(rows=1 << 40, cols=1 << 12, ld=1 << 12, ct=FAKE + 3 * G, st=FAKE + 4 * G) == N.E_SIZE     # 2^38 tiles
    assert call(rows=1 << 40, cols=1 << 12, ld=1 << 12, tile=1) == N.E_SIZE
    assert call(c=FAKE + 4080) == N.E_ALIAS                          # inside src's 4096 bytes
    assert call(s=FAKE + G + 1023) == N.E_ALIAS                      # the codes' last byte
    assert call(ct=FAKE + G, st=FAKE + 3 * G) == N.E_ALIAS
    assert call(s=FAKE + G + 1024 - 2, tile=1) == N.E_ALIAS
    assert call(rows=0) == N.OK and call(cols=0, ld=0, c=0, s=0) == N.OK


def test_gathers_refuse():
    L = N.lib()
    c = [FAKE, FAKE + G]
    s = [FAKE + 2 * G, FAKE + 3 * G]
    out = FAKE + 4 * G

    def call(c=c, s=s, world=2, S=256, dt=N.BF16, out=out):
        return L.fsdp_fp8_gather(N.ptr_array(c), N.ptr_array(s), world, S, dt, vp(out), None)

    assert call(world=0) == N.E_INVAL and call(world=129) == N.E_INVAL
    assert call(S=-1) == N.E_INVAL and call(S=1 << 62) == N.E_SIZE
    assert call(dt=9) == N.E_DTYPE and call(out=0) == N.E_INVAL
    assert call(c=[FAKE, 0]) == N.E_INVAL and call(s=[0, s[1]]) == N.E_INVAL
    assert call(c=[FAKE + 8, c[1]]) == N.E_INVAL
    assert call(out=s[1] - 1023) == N.E_ALIAS and call(out=c[0] + 254) == N.E_ALIAS and call(S=0) == N.OK

    def packed(c=c, s=s, S=256, fc=out, fs=FAKE + 5 * G):
        return L.fsdp_fp8_gather_packed(N.ptr_array(c), N.ptr_array(s), 2, S, vp(fc), vp(fs), None)

    assert packed(S=257) == N.E_SIZE and "multiple" in L.fsdp_last_error().decode()
    assert packed(fc=0) == N.E_INVAL and packed(fs=0) == N.E_INVAL and packed(fc=out + 4) == N.E_INVAL
    assert packed(c=[0, c[1]]) == N.E_INVAL and packed(c=[FAKE + 4, c[1]]) == N.E_INVAL
    assert packed(c=[out + 256, c[1]]) == N.E_ALIAS                  # shard 0 in the slot of shard 1
    assert packed(fs=out + 511) == N.E_ALIAS
    assert packed(S=0) == N.OK


def test_matmul_refuses():
    L = N.lib()
    need = L.fsdp_fp8_matmul_workspace(32, 64, 300)
    assert need >= 0
    assert L.fsdp_fp8_matmul_workspace(-1, 5, 5) == -1 and L.fsdp_fp8_matmul_workspace(1, 1, (1 << 22) + 1) == -1

    def call(a=FAKE, sa=FAKE + G, ta=0, b=FAKE + 2 * G, sb=FAKE + 3 * G, tb=0, m=32, n=64, k=300, dt=N.F32,
             out=FAKE + 4 * G, ldo=64, ws=FAKE + 5 * G, nbytes=need):
        return L.fsdp_fp8_matmul(vp(a), vp(sa), ta, vp(b), vp(sb), tb, m, n, k, dt, vp(out), ldo, vp(ws), nbytes, None)

    assert call(dt=3) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(n=-1) == N.E_INVAL and call(k=-1) == N.E_INVAL
    assert call(ldo=63) == N.E_INVAL and call(out=0) == N.E_INVAL
    assert call(a=0) == N.E_INVAL and call(sb=0) == N.E_INVAL
    assert call(a=FAKE + 4) == N.E_INVAL and call(b=FAKE + 2 * G + 8) == N.E_INVAL
    assert call(k=(1 << 22) + 1) == N.E_SIZE
    assert call(m=1 << 40, n=1 << 40, ldo=1 << 40) == N.E_SIZE
    assert call(out=FAKE + 32 * 384 - 4) == N.E_ALIAS                # A's last codes
    assert call(out=FAKE + G + 95) == N.E_ALIAS                      # A's last scale
    assert call(out=FAKE + 3 * G + 2, tb=1) == N.E_ALIAS             # B's last, in tiles: three of them
    if need:
        assert call(nbytes=need - 1) == N.E_SIZE and call(ws=0) == N.E_INVAL and call(ws=FAKE + 5 * G + 8) == N.E_INVAL
    assert call(m=0) == N.OK and call(n=0, ldo=0) == N.OK


def test_linear_refuses():
    L = N.lib()
    ws = FAKE + 5 * G
    need = L.fsdp_fp8_linear_workspace(40, 64, 300)
    assert need >= 0

    def call(x=FAKE, xdt=N.BF16, m=40, k=300, ldx=300, w=FAKE + G, sw=FAKE + 2 * G, tw=0, n=64, dt=N.F16,
             out=FAKE + 3 * G, ldo=64, ws=ws, nbytes=1 << 20):
        return L.fsdp_fp8_linear(vp(x), xdt, m, k, ldx, vp(w), vp(sw), tw, n, dt, vp(out), ldo, vp(ws), nbytes, None)

    assert call(xdt=3) == N.E_DTYPE and call(dt=-1) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(k=-1) == N.E_INVAL and call(n=-1) == N.E_INVAL
    assert call(ldx=299) == N.E_INVAL and call(ldo=63) == N.E_INVAL
    assert call(x=0) == N.E_INVAL and call(w=0) == N.E_INVAL and call(sw=0) == N.E_INVAL and call(out=0) == N.E_INVAL
    assert call(w=FAKE + G + 1) == N.E_INVAL
    assert call(k=(1 << 22) + 1, ldx=1 << 23) == N.E_SIZE
    assert call(out=FAKE + 700) == N.E_ALIAS and call(out=FAKE + 2 * G + 190) == N.E_ALIAS
    if need:
        assert call(nbytes=need - 1) == N.E_SIZE and call(ws=0) == N.E_INVAL and call(ws=ws + 8) == N.E_INVAL
        assert call(ws=FAKE + 1024) == N.E_ALIAS and call(ws=FAKE + 3 * G + 16) == N.E_ALIAS
    assert L.fsdp_fp8_linear_workspace(-1, 5, 5) == -1 and L.fsdp_fp8_linear_workspace(1 << 40, 5, 1 << 40) == -1
    assert call(m=0) == N.OK and call(n=0, ldo=0) == N.OK


def test_linear_grads_refuses():
    L = N.lib()

    def call(dy=FAKE, dydt=N.BF16, lddy=64, x=FAKE + G, xdt=N.BF16, ldx=300, m=40, n=64, k=300, wt=FAKE + 2 * G,
             swt=FAKE + 3 * G, tw=0, dxdt=N.BF16, dx=FAKE + 4 * G, lddx=300, dwdt=N.F32, dw=FAKE + 5 * G, lddw=300,
             ws=FAKE + 6 * G, nbytes=1 << 20):
        return L.fsdp_fp8_linear_grads(vp(dy), dydt, lddy, vp(x), xdt, ldx, m, n, k, vp(wt), vp(swt), tw, dxdt, vp(dx),
                                       lddx, dwdt, vp(dw), lddw, vp(ws), nbytes, None)

    assert call(dydt=5) == N.E_DTYPE and call(xdt=5) == N.E_DTYPE and call(dxdt=5) == N.E_DTYPE
    assert call(dwdt=5) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(n=-1) == N.E_INVAL and call(k=-1) == N.E_INVAL
    assert call(lddy=63) == N.E_INVAL and call(ldx=299) == N.E_INVAL and call(lddx=299) == N.E_INVAL
    assert call(lddw=299) == N.E_INVAL
    assert call(dy=0) == N.E_INVAL and call(x=0) == N.E_INVAL and call(wt=0) == N.E_INVAL and call(swt=0) == N.E_INVAL
    assert call(wt=FAKE + 2 * G + 8) == N.E_INVAL and call(ws=0) == N.E_INVAL and call(ws=FAKE + 6 * G + 4) == N.E_INVAL
    need = L.fsdp_fp8_linear_grads_workspace(40, 64, 300, 1, 1)
    assert need >= (40 + 64 + 300) * 129
    assert call(nbytes=need - 1) == N.E_SIZE
    assert 40 * 129 <= L.fsdp_fp8_linear_grads_workspace(40, 64, 300, 1, 0) < need
    assert L.fsdp_fp8_linear_grads_workspace(40, -64, 96, 1, 0) == -1
    assert call(dx=FAKE + 64) == N.E_ALIAS and call(dw=FAKE + 4 * G + 64) == N.E_ALIAS
    assert call(ws=FAKE + 5 * G + 1024) == N.E_ALIAS and call(ws=FAKE + 3 * G) == N.E_ALIAS
    assert call(m=1 << 24, lddy=64) == N.E_SIZE                          # dw sums over more than 2^22 tokens
    assert call(dx=0, dw=0, dy=0) == N.OK and call(k=0, ldx=0, lddx=0, lddw=0) == N.OK


def test_norm_refuses():
    L = N.lib()

    def call(x=FAKE, xdt=N.BF16, ldx=300, r=FAKE + G, hdt=N.F32, ldr=300, m=40, d=300, w=FAKE + 2 * G, wdt=N.F32,
             eps=1e-6, h=FAKE + 3 * G, ldh=300, ydt=N.F32, y=0, ldy=300, c=FAKE + 5 * G, s=FAKE + 6 * G,
             rstd=FAKE + 7 * G):
        return L.fsdp_rms_norm_fp8(vp(x), xdt, ldx, vp(r), hdt, ldr, m, d, vp(w), wdt, eps, vp(h), ldh, ydt, vp(y), ldy,
                                   vp(c), vp(s), vp(rstd), None)

    assert call(xdt=3) == N.E_DTYPE and call(hdt=3) == N.E_DTYPE and call(wdt=3) == N.E_DTYPE
    assert call(ydt=3, y=FAKE + 4 * G) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(d=-1) == N.E_INVAL
    assert call(d=N.RMS_MAX_D + 1, ldx=1 << 16, ldr=1 << 16, ldh=1 << 16) == N.E_SIZE and call(m=1 << 60) == N.E_SIZE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == N.E_INVAL
    assert call(ldx=299) == N.E_INVAL and call(ldr=299) == N.E_INVAL and call(ldh=299) == N.E_INVAL
    assert call(y=FAKE + 4 * G, ldy=299) == N.E_INVAL
    assert call(x=0) == N.E_INVAL and call(w=0) == N.E_INVAL and call(c=0) == N.E_INVAL and call(s=0) == N.E_INVAL
    assert call(r=0) == N.E_INVAL and call(h=0) == N.E_INVAL             # they come together
    assert call(c=FAKE + 5 * G + 8) == N.E_INVAL and call(rstd=FAKE + 7 * G + 2) == N.E_INVAL
    # h may be the residual, but not a shifted one, nor an x of another size
    assert call(h=FAKE + G + 4) == N.E_ALIAS and call(h=FAKE + G, ldh=304) == N.E_ALIAS
    assert call(h=FAKE) == N.E_ALIAS
    assert call(y=FAKE, ydt=N.BF16) == N.E_ALIAS and call(y=FAKE + 3 * G) == N.E_ALIAS
    assert call(c=FAKE + 1024) == N.E_ALIAS and call(s=FAKE + 5 * G + 40 * 384 - 1) == N.E_ALIAS
    assert call(rstd=FAKE + 2 * G + 1196) == N.E_ALIAS and call(h=FAKE + 2 * G) == N.E_ALIAS
    assert call(m=0) == N.OK and call(d=0, ldx=0, ldr=0, ldh=0) == N.OK


def test_norm_grads_refuses():
    L = N.lib()
    need = L.fsdp_rms_norm_grads_workspace(40, 300, 1)
    assert need >= 300 * 4 and L.fsdp_rms_norm_grads_workspace(40, 300, 0) == 0
    assert L.fsdp_rms_norm_grads_workspace(1, 300, 1) == 0 and L.fsdp_rms_norm_grads_workspace(0, 300, 1) == 0
    assert L.fsdp_rms_norm_grads_workspace(-1, 300, 1) == -1 and L.fsdp_rms_norm_grads_workspace(1, 1 << 16, 1) == -1

    def call(dy=FAKE, ydt=N.BF16, lddy=300, h=FAKE + G, hdt=N.F32, ldh=300, m=40, d=300, w=FAKE + 2 * G, wdt=N.F32,
             rstd=FAKE + 3 * G, dh=FAKE + 4 * G, lddh=300, dx=FAKE + 5 * G, lddx=300, dwdt=N.F32, dw=FAKE + 6 * G,
             ws=FAKE + 7 * G, nbytes=need):
        return L.fsdp_rms_norm_grads(vp(dy), ydt, lddy, vp(h), hdt, ldh, m, d, vp(w), wdt, vp(rstd), vp(dh), lddh,
                                     vp(dx), lddx, dwdt, vp(dw), vp(ws), nbytes, None)

    assert call(ydt=3) == N.E_DTYPE and call(hdt=3) == N.E_DTYPE and call(wdt=3) == N.E_DTYPE
    assert call(dwdt=3) == N.E_DTYPE
    assert call(m=-1) == N.E_INVAL and call(d=-1) == N.E_INVAL
    assert call(d=N.RMS_MAX_D + 1, lddy=1 << 16, ldh=1 << 16, lddh=1 << 16, lddx=1 << 16) == N.E_SIZE
    assert call(lddy=299) == N.E_INVAL and call(ldh=299) == N.E_INVAL and call(lddh=299) == N.E_INVAL
    assert call(lddx=299) == N.E_INVAL
    assert call(dy=0) == N.E_INVAL and call(h=0) == N.E_INVAL and call(w=0) == N.E_INVAL and call(rstd=0) == N.E_INVAL
    assert call(rstd=FAKE + 3 * G + 1) == N.E_INVAL
    assert call(nbytes=need - 1) == N.E_SIZE and call(ws=0) == N.E_INVAL and call(ws=FAKE + 7 * G + 8) == N.E_INVAL
    assert call(dx=FAKE + 4 * G + 4) == N.E_ALIAS and call(dx=FAKE) == N.E_ALIAS and call(dx=FAKE + G) == N.E_ALIAS
    assert call(dw=FAKE + 5 * G) == N.E_ALIAS and call(dw=FAKE + 2 * G) == N.E_ALIAS and call(ws=FAKE + 6 * G) == N.E_ALIAS
    assert call(dx=0, dw=0) == N.OK and call(m=0, dw=0) == N.OK and call(d=0, lddy=0, ldh=0, lddh=0, lddx=0) == N.OK


def test_binding_refuses():
    z = torch.zeros(4, 64)
    for f in (lambda: ss.fsdp_fp8_quantize(z), lambda: ss.fsdp_fp8_quantize(z, form="diagonal"),
              lambda: ss.fsdp_fp8_quantize(z, out_t=1), lambda: ss.fsdp_fp8_gather([]),
              lambda: ss.fsdp_fp8_gather([z]), lambda: ss.fsdp_rms_norm_fp8(z, z[0]),
              lambda: ss.fsdp_rms_norm_grads(z, z, z[0], z[:, 0])):
        with pytest.raises(ValueError):
            f()
    a = ss.Fp8.empty(4, 200, "cpu")
    assert a.shape == (4, 200) and a.codes.shape == (4, 256) and a.scales.shape == (4, 2)
    t = ss.Fp8.empty(130, 200, "cpu", tile=True)
    assert t.scales.shape == (2, 2) and "tiles" in repr(t)
    for f in (lambda: ss.Fp8(a.codes, a.scales, 128),                # one block, not two
              lambda: ss.Fp8(a.codes[:, :128], a.scales[:, :1], 128),    # rows not next to each other
              lambda: ss.Fp8(a.codes, a.scales[:2], 200),
              lambda: ss.Fp8(t.codes, t.scales, 200),                # tiles that are not said to be
              lambda: ss.Fp8(a.codes, a.scales, 200, tile=True),
              lambda: ss.Fp8(a.codes.view(-1)[4:].view(-1)[:512].view(2, 256), a.scales[:2], 200),
              lambda: ss.fsdp_fp8_matmul(a, a),                      # on the host
              lambda: ss.fsdp_fp8_linear(torch.zeros(2, 200), a),
              lambda: ss.fsdp_fp8_views(t, [(1,)])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ss.fsdp_fp8_linear(torch.zeros(2, 64), z), lambda: ss.fsdp_fp8_matmul(z, a)):
        with pytest.raises(TypeError):
            f()


def test_views_of_a_packed_unit():
    full = ss.Fp8.empty(1, 128 * 40, "cpu")
    full.scales.copy_(torch.arange(40, dtype=torch.uint8).view(1, 40))
    v = ss.fsdp_fp8_views(full, [(128,), (4, 256), (5,), (3, 128), (123,), (2, 2, 128)])
    assert [x.shape if x is not None else None for x in v] == [(1, 128), (4, 256), None, None, None, (4, 128)]
    assert v[1].scales.tolist() == [[1, 2], [3, 4], [5, 6], [7, 8]]
    # 128 + 1024 + 5 + 384 + 123 = 1664 elements lie before the last tensor
    assert v[5].codes.data_ptr() == full.codes.data_ptr() + 1664 and v[5].scales[0, 0] == 13
    with pytest.raises(ValueError):
        ss.fsdp_fp8_views(full, [(41, 128)])


@pytest.mark.parametrize("tile", [False, True])
def test_copies_have_memory_of_their_own(tile):
    q = ss.Fp8.empty(130, 300, "cpu", tile)
    q.codes.copy_(torch.arange(q.codes.numel()).view_as(q.codes) % 120)
    q.scales.fill_(127)
    for same in (copy.deepcopy(q), pickle.loads(pickle.dumps(q)), ss.Fp8(q.codes.clone(), q.scales.clone(), 300, tile)):
        assert same.shape == (130, 300) and same.tile == tile and same.device == q.device
        assert torch.equal(same.codes, q.codes) and torch.equal(same.scales, q.scales)
        assert same._ptrs() == (same.codes.data_ptr(), same.scales.data_ptr())
        assert not set(same._ptrs()) & set(q._ptrs())
        same.codes.zero_()
        assert q.codes.any()
    fresh = copy.deepcopy(ss.Fp8.empty(3, 128, "cpu", tile))     # before anybody asked for its views
    assert fresh._ptrs() == (fresh.codes.data_ptr(), fresh.scales.data_ptr())
