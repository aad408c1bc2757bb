"""The gradient norm and clipping on the host: argument validation of the C
entry points (before anything touches the device: fake, never-dereferenced
pointers reach every check) and of the binding."""
import ctypes
import math

import pytest
import torch

import sharded_state_amd as ss
from sharded_state_amd import _native as N

FAKE = 1 << 40
WS = FAKE + (1 << 36)
OUT = FAKE + (1 << 37)


def vp(x):
    return ctypes.c_void_p(x)


def i32_array(vals):
    return (ctypes.c_int32 * max(len(vals), 1))(*vals)


def _norm(ptrs, numels, dts, n=None, max_norm=1.0, outs=(OUT, OUT + 8, OUT + 12), ws=WS):
    return N.lib().fsdp_grad_norm(N.ptr_array(ptrs), N.i64_array(numels), i32_array(dts),
                                  len(ptrs) if n is None else n, max_norm, vp(outs[0]), vp(outs[1]), vp(outs[2]),
                                  vp(ws), None)


def test_grad_norm_refuses():
    a = FAKE
    assert _norm([a], [10], [7]) == N.E_DTYPE
    assert _norm([a], [-1], [N.F32]) == N.E_INVAL
    assert _norm([0], [10], [N.F32]) == N.E_INVAL
    assert _norm([a], [10], [N.F32], n=-1) == N.E_INVAL
    assert _norm([a], [10], [N.F32], outs=(0, 0, 0)) == N.E_INVAL
    assert _norm([a], [10], [N.F32], ws=0) == N.E_INVAL
    assert _norm([a], [10], [N.F32], ws=WS + 4) == N.E_INVAL
    assert _norm([a], [10], [N.F32], outs=(OUT + 4, 0, 0)) == N.E_INVAL
    assert _norm([a], [10], [N.F32], outs=(OUT, OUT + 10, 0)) == N.E_INVAL
    for bad in (-1.0, math.inf, math.nan):
        assert _norm([a], [10], [N.F32], max_norm=bad) == N.E_INVAL
    assert _norm([OUT - 36], [10], [N.F32]) == N.E_ALIAS            # the sum would land in the tensor
    assert _norm([WS + 32764], [10], [N.F32]) == N.E_ALIAS          # the workspace's last bytes
    assert _norm([a], [10], [N.F32], outs=(WS + 8, 0, 0)) == N.E_ALIAS
    assert _norm([a], [10], [N.F32], outs=(OUT, OUT + 4, 0)) == N.E_ALIAS
    assert _norm([a], [(1 << 63) - 1], [N.BF16]) == N.E_SIZE
    big = (1 << 62) // 16
    assert _norm([a] * 16, [big] * 16, [N.BF16] * 16) == N.E_SIZE
    assert "too large" in N.lib().fsdp_last_error().decode()


def test_grad_norm_units_refuses():
    L = N.lib()
    g = N.ptr_array([FAKE, FAKE + (1 << 30)])

    def call(units, n=None, world=2, rank=0, gdt=N.F16, max_norm=1.0, outs=(OUT, OUT + 8, OUT + 12), ws=WS):
        t = (N.NormUnit * max(len(units), 1))(*units)
        return L.fsdp_grad_norm_units(t, len(units) if n is None else n, world, rank, gdt, 1, max_norm, vp(outs[0]),
                                      vp(outs[1]), vp(outs[2]), vp(ws), None)

    unit = N.NormUnit(g, None, 1000)
    assert call([unit], world=0) == N.E_INVAL
    assert call([unit], world=129) == N.E_INVAL
    assert call([unit], rank=2) == N.E_INVAL
    assert call([unit], gdt=5) == N.E_DTYPE
    assert call([unit], n=-1) == N.E_INVAL
    assert call([N.NormUnit(g, None, -1)]) == N.E_INVAL
    assert call([N.NormUnit(N.ptr_array([FAKE, 0]), None, 10)]) == N.E_INVAL
    assert call([N.NormUnit(g, FAKE + 1000, 1000)]) == N.E_ALIAS          # the shard over a gradient block
    assert call([N.NormUnit(g, WS, 1000)]) == N.E_ALIAS
    s = FAKE + (1 << 34)
    assert call([N.NormUnit(g, s, 1000), N.NormUnit(g, s + 3996, 1000)]) == N.E_ALIAS
    assert call([unit], ws=0) == N.E_INVAL
    assert call([unit], max_norm=math.nan) == N.E_INVAL
    assert call([N.NormUnit(g, None, 1 << 62)]) == N.E_SIZE


def test_combine_refuses():
    L = N.lib()
    assert L.fsdp_grad_norm_combine(vp(FAKE), -1, 1.0, None, vp(OUT), None, None) == N.E_INVAL
    assert L.fsdp_grad_norm_combine(None, 2, 1.0, None, vp(OUT), None, None) == N.E_INVAL
    assert L.fsdp_grad_norm_combine(vp(FAKE + 4), 2, 1.0, None, vp(OUT), None, None) == N.E_INVAL
    assert L.fsdp_grad_norm_combine(vp(FAKE), 2, 1.0, vp(FAKE + 8), None, None, None) == N.E_ALIAS
    assert L.fsdp_grad_norm_combine(vp(FAKE), 2, -1.0, None, None, vp(OUT), None) == N.E_INVAL
    assert L.fsdp_grad_norm_combine(vp(FAKE), 2, 1.0, None, None, None, None) == N.E_INVAL


def test_clip_refuses():
    L = N.lib()

    def call(ptrs, numels, dts, coef=OUT):
        return L.fsdp_clip_grads(N.ptr_array(ptrs), N.i64_array(numels), i32_array(dts), len(ptrs), vp(coef), None)

    assert call([FAKE], [10], [N.F32], coef=0) == N.E_INVAL
    assert call([FAKE], [10], [N.F32], coef=OUT + 2) == N.E_INVAL
    assert call([FAKE], [10], [3]) == N.E_DTYPE
    assert call([0], [10], [N.F32]) == N.E_INVAL
    assert call([FAKE, FAKE], [10, 10], [N.F32, N.F32]) == N.E_ALIAS     # the same tensor twice
    assert call([FAKE, FAKE + 18], [10, 10], [N.F16, N.F16]) == N.E_ALIAS
    assert call([OUT - 36], [10], [N.F32]) == N.E_ALIAS                  # the coefficient inside the tensor
    assert call([0, 0], [0, 0], [N.F32, N.BF16]) == N.OK                 # nothing to scale: no device work
    assert call([], [], []) == N.OK


def test_step_clipped_refuses():
    L = N.lib()
    hp = ss.OptimHP.adamw()
    a = FAKE
    g = N.ptr_array([FAKE + (4 << 30), FAKE + (5 << 30)])
    unit = N.Unit(a, a + (1 << 30), a + (2 << 30), g, None, None, a + (3 << 30), 1000)

    def call(coef, hp=hp):
        t = (N.Unit * 1)(unit)
        return L.fsdp_step_units_clipped(t, 1, 2, 0, N.F16, 1, N.F32, N.F16, ctypes.byref(hp), vp(coef), None)

    assert call(0) == N.E_INVAL and "coef" in L.fsdp_last_error().decode()
    assert call(OUT + 1) == N.E_INVAL
    assert call(a + 400) == N.E_ALIAS                                    # the coefficient inside the master shard
    assert call(OUT, ss.OptimHP.adamw(step=0)) == N.E_INVAL


def test_binding_refuses():
    with pytest.raises(ValueError):
        ss.fsdp_grad_norm([torch.zeros(4)])                              # a host tensor
    for bad in (3.0, None, [torch.zeros(4)]):
        with pytest.raises(TypeError):
            ss.fsdp_grad_norm([bad])                                     # no tensor
    with pytest.raises(ValueError):
        ss.fsdp_grad_norm([torch.zeros(4, dtype=torch.int32)])
    with pytest.raises(ValueError):
        ss.fsdp_grad_norm([])
    with pytest.raises(ValueError):
        ss.fsdp_grad_norm_units([], 0, True)
    for bad in (-1.0, math.inf, math.nan):
        with pytest.raises(ValueError):
            ss.fsdp_grad_norm_units([dict()], 0, True, max_norm=bad)
    with pytest.raises(ValueError):
        ss.fsdp_clip_grads([], torch.ones(1))
    gn = ss.GradNorm("cpu")
    assert gn.coef is None and gn.sumsq.dtype == torch.float64 and gn.norm.numel() == 1
    with pytest.raises(ValueError):
        ss.fsdp_clip_grads([], gn)                                       # taken without max_norm
    with pytest.raises(ValueError):
        ss.fsdp_grad_norm([], out=gn)                                    # host memory
