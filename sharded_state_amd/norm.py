"""The global gradient norm and clipping, between the backward and the step.

Clipping keeps the norm over every gradient of a model at or under a bound by
one factor for all of them:

    q = sum of x^2 (64 bits),  norm = sqrt(q),  coef = min(1, max_norm / (norm + 1e-6))

``fsdp_grad_norm`` takes a list of gradient tensors, ``fsdp_grad_norm_units`` a
rank's units as ``fsdp_step_units`` has them (the averaged gradient of its
shards, reduced on the way and stored where wanted).  Nothing comes back to the
host: ``fsdp_clip_grads`` and ``fsdp_step_units(..., clip=...)`` read the
coefficient on the device.  A job of N processes adds the ranks' ``sumsq`` (one
all-reduce of one double) and takes the norm of the whole from
``fsdp_grad_norm_combine``.

A norm that is not finite is applied as the formula says: an infinite one gives
coefficient 0, a NaN one gives NaN.  A loop that wants to skip such a step reads
``norm`` before it steps.  A norm taken without max_norm leaves the coefficient
of the largest bound in its GradNorm: 1 for every finite norm, so a prepared or
captured step that reads it is not clipped by an earlier norm.
"""
import ctypes
import sys
from array import array

import torch

from . import _native as N
from ._native import ptr_array
from .api import _DT, _dev, _grads, _issue, _on, _same_device, dtype_code

_WS = N.NORM_WORKSPACE_BYTES


class GradNorm:
    """Where a norm call writes: one device allocation with the sum of squares,
    the norm, the clipping coefficient and the call's workspace.

    sumsq  float64, 1 element;  norm  float32, 1 element
    coef   float32, 1 element (None if the last call had no max_norm; what a
           step prepared with this object then reads is 1, or 0 and NaN by the
           formula where the norm is infinite or NaN)

    Calls that may run at the same time, replays of two captured graphs among
    them, need a GradNorm each."""

    def __init__(self, device="cuda"):
        self._buf = torch.empty(16 + _WS, dtype=torch.uint8, device=device)
        self.has_coef = False

    @property
    def device(self):
        return self._buf.device

    @property
    def sumsq(self):
        return self._buf[:8].view(torch.float64)

    @property
    def norm(self):
        return self._buf[8:12].view(torch.float32)

    @property
    def coef(self):
        return self._buf[12:16].view(torch.float32) if self.has_coef else None

    def _issue(self, name, stream, args, max_norm, workspace=True):
        """Issue a norm call whose outputs are this object's."""
        p = self._buf.data_ptr()
        clips = max_norm is not None
        # the coefficient is always written: a prepared step may read it at any later issue
        args += (float(max_norm) if clips else sys.float_info.max, p, p + 8, p + 12)
        _issue(name, self.device, stream, *args, *((p + 16,) if workspace else ()))
        self.has_coef = clips
        return self


def _out(out, device, stream):
    if out is None:
        with _on(stream):
            return GradNorm(device)
    if not isinstance(out, GradNorm):
        raise TypeError("out must be a GradNorm")
    if out.device.type != "cuda":
        raise ValueError("out must be on a device, got %s" % out.device)
    if out.device != device:
        raise ValueError("out is on %s, the gradients on %s" % (out.device, device))
    return out


def _max_norm(max_norm):
    if max_norm is not None and not 0.0 <= float(max_norm) < float("inf"):
        raise ValueError("max_norm must be finite and >= 0, got %r" % (max_norm,))


def clip_coef(clip):
    """The device coefficient of `clip`: a GradNorm with one, or a float32
    tensor of one element."""
    if isinstance(clip, GradNorm):
        if not clip.has_coef:
            raise ValueError("the norm was taken without max_norm: it has no clipping coefficient")
        return clip.coef
    _dev(clip, "clip")
    if clip.dtype != torch.float32 or clip.numel() != 1:
        raise ValueError("clip must be a GradNorm or one float32 element")
    return clip


def _host(ctype, code, values):
    """`values` as a host array of ctype (one element where there are none).  A
    long list goes through an array: an element's conversion costs less there, the
    array itself 0.6 us."""
    n = len(values)
    if n < 16:
        return (ctype * max(n, 1))(*values)
    return (ctype * n).from_buffer(array(code, values))


def _list(tensors, name):
    """A list of contiguous tensors on one device, with its host arrays.  The
    checks are a pass each over the whole list, and the tensors are looked at one
    by one only to say what is wrong: a model has hundreds of them."""
    tensors = list(tensors)
    try:
        devices = {t.get_device() for t in tensors}              # -1: not on a device
        whole = all([t.is_contiguous() for t in tensors])
        codes = [_DT[t.dtype] for t in tensors]
    except (AttributeError, KeyError):
        devices, whole, codes = {-1}, False, []
    if not whole or -1 in devices or len(devices) > 1:
        for i, t in enumerate(tensors):
            dtype_code(_dev(t, "%s[%d]" % (name, i)).dtype)
        _same_device(tensors)
    return (tensors, _host(ctypes.c_void_p, "q", [t.data_ptr() for t in tensors]),
            _host(ctypes.c_int64, "q", [t.numel() for t in tensors]), _host(ctypes.c_int32, "i", codes), len(tensors))


def fsdp_grad_norm(tensors, max_norm=None, out=None, stream=None):
    """Norm over a list of gradient tensors (any mix of float32, float16 and
    bfloat16, each contiguous); with max_norm the clipping coefficient too.
    Returns the GradNorm (`out`, or a new one)."""
    tensors, ptrs, numels, dts, n = _list(tensors, "tensors")
    _max_norm(max_norm)
    if not tensors and out is None:
        raise ValueError("no tensors and no out: nothing says which device to use")
    device = tensors[0].device if tensors else out.device
    out = _out(out, device, stream)
    return out._issue("fsdp_grad_norm", stream, (ptrs, numels, dts, n), max_norm)


def fsdp_grad_norm_units(units, rank, fp32_reduce, max_norm=None, out=None, stream=None):
    """Norm over rank `rank`'s shards of the averaged gradient of `units`, in the
    pass that reduces them.  A unit is a dict as fsdp_step_units has it:
    rank_grads, and master or shard_numel for the shard's size; with grad_shard
    (of that size, the dtype of fsdp_reduce_scatter_local) the averaged shard is
    stored there.
    All units share world, rank and dtype.  Returns the GradNorm."""
    _max_norm(max_norm)
    if not units:
        raise ValueError("units is empty")
    world = len(units[0]["rank_grads"])
    table = (N.NormUnit * len(units))()
    keep, tensors, gdt = [], [], None
    for k, u in enumerate(units):
        shard, S = u.get("grad_shard"), u.get("shard_numel")
        if S is not None:
            S = int(S)
        for t in (shard, u.get("master")):
            if t is None:
                continue
            if S is None:
                S = t.numel()
            elif t.numel() != S:                 # rank r's block of a gradient begins at r * S
                raise ValueError("units[%d]: grad_shard, master and shard_numel give the sizes %d and %d"
                                 % (k, S, t.numel()))
        if S is None:
            raise ValueError("units[%d] needs grad_shard, master or shard_numel" % k)
        grads, w, g_dt = _grads(u["rank_grads"], S)
        if w != world:
            raise ValueError("units[%d] has %d ranks, units[0] %d" % (k, w, world))
        gdt = gdt or g_dt
        if g_dt != gdt:
            raise TypeError("every unit's gradients must share one dtype")
        if shard is not None:
            _dev(shard, "units[%d].grad_shard" % k)
            odt = torch.float32 if (fp32_reduce or gdt == torch.float32) else gdt
            if shard.dtype != odt:
                raise TypeError("units[%d].grad_shard must be %s" % (k, odt))
            tensors.append(shard)
        tensors += grads
        gptr = ptr_array([g.data_ptr() for g in grads])
        keep.append(gptr)
        table[k] = N.NormUnit(gptr, shard.data_ptr() if shard is not None else None, S)
    _same_device(tensors)
    device = tensors[0].device
    out = _out(out, device, stream)
    return out._issue("fsdp_grad_norm_units", stream, (table, len(units), world, int(rank), dtype_code(gdt),
                                                       int(bool(fp32_reduce))), max_norm)


def fsdp_grad_norm_combine(sumsqs, max_norm=None, out=None, stream=None):
    """Norm (and coefficient) of the ranks' sums of squares: a float64 device
    tensor of their `sumsq`, added in order."""
    _dev(sumsqs, "sumsqs")
    _max_norm(max_norm)
    if sumsqs.dtype != torch.float64:
        raise TypeError("sumsqs must be float64")
    device = sumsqs.device
    out = _out(out, device, stream)
    return out._issue("fsdp_grad_norm_combine", stream, (sumsqs.data_ptr(), sumsqs.numel()), max_norm, workspace=False)


def fsdp_clip_grads(tensors, clip, stream=None):
    """Scale every tensor in place by the coefficient of `clip` (a GradNorm, or
    one float32 element on the device): an fp32 product rounded to the tensor's
    dtype.  A coefficient of exactly 1 leaves them untouched."""
    tensors, ptrs, numels, dts, n = _list(tensors, "tensors")
    coef = clip_coef(clip)
    _same_device(tensors[:1] + [coef])
    device = coef.device
    _issue("fsdp_clip_grads", device, stream, ptrs, numels, dts, n, coef.data_ptr())
    return tensors
