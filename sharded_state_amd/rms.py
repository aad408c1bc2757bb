"""The root-mean-square norm over features in front of an 8-bit product: the
residual's addition before it, 8-bit blocks behind it, and its gradients.

    o = ss.fsdp_rms_norm_fp8(x, weight, residual)          # o.h = x + residual, o.q its norm in blocks
    y = ss.fsdp_fp8_linear(o.q, w)
    dx, dw = ss.fsdp_rms_norm_grads(dy, o.h, weight, o.rstd, dh=dh)

dx is the gradient of x and of the residual alike; dh is the gradient that the
sum has from elsewhere, the residual path behind the layer.  A tensor given for a result
counts as changed in place: a graph that saved it refuses its backward.
"""
import collections

import torch

from . import _native as N
from .api import _changed, _issue, _no_tangents, _on, dtype_code
from .fp8 import Fp8, _target
from .mx4 import _matrix, _one_device, _result, _space

RmsNorm = collections.namedtuple("RmsNorm", "q h rstd y")
RmsNorm.__doc__ = """What fsdp_rms_norm_fp8 gives: the normed rows in 8-bit blocks (Fp8), the sum h that
they are the norm of, rstd (float32, one a row), and the normed rows as a tensor (None
unless asked for)."""


def _rows(t, name, m=None, d=None):
    """(rows, columns, row stride) of a matrix; of m x d where they are given."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    r = _matrix(t, name)
    if m is not None and r[:2] != (m, d):
        raise ValueError("%s must be a matrix of %d x %d" % (name, m, d))
    return r


def _vector(n, dtype, device, stream):
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(n, dtype=dtype, device=device)


def _features(t, name, d, device):
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.shape[0] != d or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d elements" % (name, d))
    _one_device(device, t)
    return t


def fsdp_rms_norm_fp8(x, weight, residual=None, eps=1e-6, out=None, h=None, y=None, stream=None):
    """h = x + residual (in the residual's dtype; x itself without one), and its
    root-mean-square norm times `weight` in 8-bit blocks, as an RmsNorm.

    x, residual  matrices [tokens, features], rows may be strided
    weight       [features], any of the dtypes and any alignment (its view in a flat unit)
    out, h       where to put the blocks (an Fp8) and the sum; h may be the residual, or an
                 x of its dtype
    y            True, or a matrix: the normed rows as a tensor too (dtype of x for True)

    Of no features rstd is NaN, the mean of nothing.

    No graph: where grad mode is on, an input that requires grad is refused, and so is one with a
    forward-mode tangent."""
    _no_tangents(x, weight, residual)
    m, d, ldx = _rows(x, "x")
    device = x.device
    _features(weight, "weight", d, device)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, residual)):
        raise ValueError("an input requires grad, and the outputs would carry none: call under torch.no_grad() or "
                         "detach it, and take the gradients from fsdp_rms_norm_grads")
    given = h, y
    res, ldr, cr, ldh = None, 0, 0, 0
    if residual is not None:
        ldr = _rows(residual, "residual", m, d)[2]
        h, ldh = _result(h, m, d, residual.dtype, device, stream)
        if h.dtype != residual.dtype:
            raise TypeError("h dtype %s differs from the residual's %s" % (h.dtype, residual.dtype))
        _one_device(device, residual, h)
        res, cr = residual.data_ptr(), dtype_code(residual.dtype)
    elif h is not None:
        raise ValueError("without a residual h is x itself")
    out = _target(out, m, d, False, device, stream, "out")
    py, cy, ldy = None, 0, 0
    if y is not None and y is not False:
        y, ldy = _result(None if y is True else y, m, d, x.dtype, device, stream)
        _one_device(device, y)
        py, cy = y.data_ptr(), dtype_code(y.dtype)
    else:
        y = None
    rstd = _vector(m, torch.float32, device, stream)
    if d == 0:                                   # the mean of nothing; the call writes nothing
        with _on(stream):
            rstd.fill_(float("nan"))
    _issue("fsdp_rms_norm_fp8", device, stream, x.data_ptr(), dtype_code(x.dtype), ldx, res, cr, ldr, m, d,
           weight.data_ptr(), dtype_code(weight.dtype), float(eps), h.data_ptr() if res is not None else None, ldh, cy,
           py, ldy, *out._ptrs(), rstd.data_ptr())
    _changed(*given)
    return RmsNorm(out, x if residual is None else h, rstd, y)


def fsdp_rms_norm_grads(dy, h, weight, rstd, dh=None, dx=None, dw=None, dw_dtype=None, stream=None):
    """Gradients of the norm from dy [tokens, features] and what the forward gave:
    dx (dtype of h; with dh, the gradient that h has from elsewhere, added to it)
    and dw (dw_dtype, else the weight's dtype).  dx and dw may be given (dx may be
    dh, or a dy of h's dtype; dw: the weight's place in a flat gradient); dx=False
    or dw=False: not wanted, and None in its place."""
    _no_tangents(dy, h, weight, rstd, dh)
    m, d, lddy = _rows(dy, "dy")
    device = dy.device
    ldh = _rows(h, "h", m, d)[2]
    _features(weight, "weight", d, device)
    _features(rstd, "rstd", m, device)
    if rstd.dtype != torch.float32:
        raise TypeError("rstd must be float32, got %s" % rstd.dtype)
    _one_device(device, h)
    want_dx, want_dw = dx is not False, dw is not False
    given = dx, dw
    pe, lde = None, 0
    if dh is not None:
        lde = _rows(dh, "dh", m, d)[2]
        if dh.dtype != h.dtype:
            raise TypeError("dh dtype %s differs from h's %s" % (dh.dtype, h.dtype))
        _one_device(device, dh)
        pe = dh.data_ptr()
    pdx = pdw = None
    lddx = cdw = 0
    if want_dx:
        dx, lddx = _result(dx, m, d, h.dtype, device, stream)
        if dx.dtype != h.dtype:
            raise TypeError("dx dtype %s differs from h's %s" % (dx.dtype, h.dtype))
        _one_device(device, dx)
        pdx = dx.data_ptr()
    if want_dw:
        if dw is None:
            dw = _vector(d, dw_dtype or weight.dtype, device, stream)
        _features(dw, "dw", d, device)
        pdw, cdw = dw.data_ptr(), dtype_code(dw.dtype)
    keep, space, nbytes = _space(N.lib().fsdp_rms_norm_grads_workspace(m, d, int(want_dw)), device, stream)
    _issue("fsdp_rms_norm_grads", device, stream, dy.data_ptr(), dtype_code(dy.dtype), lddy, h.data_ptr(),
           dtype_code(h.dtype), ldh, m, d, weight.data_ptr(), dtype_code(weight.dtype), rstd.data_ptr(), pe, lde, pdx,
           lddx, cdw, pdw, space, nbytes)
    _changed(*given)
    return dx if want_dx else None, dw if want_dw else None
