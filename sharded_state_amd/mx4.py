"""4-bit microscaled blocks: the compute copy at 17/32 byte an element, its
all-gather, and products of matrices kept that way.

Blocks of 32 elements share a power of two; an element is a sign and one of
0, 0.5, 1, 1.5, 2, 3, 4, 6 (include/fsdp_shard.h has the format to the bit).

    mine = ss.fsdp_mx4_quantize(master)                    # this rank's shard
    full = ss.fsdp_mx4_gather(shards, full)                # N shards -> the 16-bit full buffer
    packed = ss.fsdp_mx4_gather_packed(shards)             # N shards -> one packed unit
    w = ss.fsdp_mx4_views(packed, shapes)[k]               # a weight of it, nothing copied
    y = ss.fsdp_mx4_linear(x, w)                           # x quantised on the way, y = x W^T

A product needs its blocks along the summed axis.  The forward sums over the
input features, the gradient of x over the output features and the gradient of
W over the tokens, so ``fsdp_mx4_linear_grads`` quantises dy and x along the
axes that it sums over and takes W quantised along its columns
(``fsdp_mx4_quantize(w, form="columns")``).  Quantisation itself is passed
through unchanged by the gradients.
"""
import torch

from . import _native as N
from ._native import ptr_array
from .api import _dev, _issue, _on, dtype_code

BLOCK = 32


def _blocks(cols):
    return -(-cols // BLOCK)


class Mx4:
    """A matrix of `rows` x `cols` in 4-bit blocks along its rows.

    codes   uint8 [rows, ceil(cols / 32) * 16], contiguous, 16-byte aligned
    scales  uint8 [rows, ceil(cols / 32)], contiguous"""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales, cols):
        nb = _blocks(cols)
        for name, t, w in (("codes", codes, nb * 16), ("scales", scales, nb)):
            if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[1] != w or not t.is_contiguous():
                raise ValueError("%s must be a contiguous uint8 matrix of %d columns for cols = %d" % (name, w, cols))
        if codes.shape[0] != scales.shape[0]:
            raise ValueError("codes has %d rows, scales %d" % (codes.shape[0], scales.shape[0]))
        if codes.device != scales.device:
            raise ValueError("codes is on %s, scales on %s" % (codes.device, scales.device))
        if codes.data_ptr() % 16:
            raise ValueError("codes must be 16-byte aligned")
        self.codes, self.scales, self.rows, self.cols = codes, scales, codes.shape[0], int(cols)

    @classmethod
    def empty(cls, rows, cols, device="cuda"):
        nb = _blocks(cols)
        self = object.__new__(cls)               # what is allocated here needs no check
        self.codes = torch.empty((rows, nb * 16), dtype=torch.uint8, device=device)
        self.scales = torch.empty((rows, nb), dtype=torch.uint8, device=device)
        self.rows, self.cols = rows, cols
        return self

    @property
    def device(self):
        return self.codes.device

    @property
    def shape(self):
        return (self.rows, self.cols)

    def __repr__(self):
        return "Mx4(%d x %d, %s)" % (self.rows, self.cols, self.device)


def _matrix(t, name):
    """A device tensor as (rows, columns, row stride); 1-D is one row."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor, got %s" % (name, t.device))
    shape = t.shape
    if len(shape) == 1:
        cols = shape[0]
        if cols > 1 and t.stride(0) != 1:
            raise ValueError("%s must have its elements next to each other" % name)
        return 1, cols, cols
    if len(shape) != 2:
        raise ValueError("%s must have one or two dimensions, got %d" % (name, len(shape)))
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1 or rows > 1 and cols > 0 and ld < cols:
        raise ValueError("%s must have its rows' elements next to each other" % name)
    return rows, cols, ld if rows > 1 else cols


def _result(out, rows, cols, dtype, device, stream):
    """A product's output, allocated where none is given, as (tensor, row stride)."""
    if out is None:
        with _on(stream):
            return torch.empty((rows, cols), dtype=dtype, device=device), cols
    if not isinstance(out, torch.Tensor) or tuple(out.shape) != (rows, cols):
        raise ValueError("out must be a matrix of %d x %d" % (rows, cols))
    return out, _matrix(out, "out")[2]


def _one_device(device, *tensors):
    for t in tensors:
        if t.device != device:
            raise ValueError("all tensors must be on one device, got %s and %s" % (device, t.device))


def _target(out, rows, cols, device, stream, name):
    if out is None:
        with _on(stream):
            return Mx4.empty(rows, cols, device)
    if not isinstance(out, Mx4):
        raise TypeError("%s must be an Mx4" % name)
    if out.shape != (rows, cols) or out.device != device:
        raise ValueError("%s must be %d x %d on %s, got %r" % (name, rows, cols, device, out))
    return out


def fsdp_mx4_quantize(src, out=None, out_t=None, form="rows", stream=None):
    """A flat shard (1-D: one row) or a matrix (2-D, its rows may be strided) of
    float32, float16 or bfloat16 in 4-bit blocks.  form "rows": blocks along the
    rows, as Mx4 of src's shape; "columns": blocks along the columns, as Mx4 of
    the transpose's shape; "both": the two of them."""
    if form not in ("rows", "columns", "both"):
        raise ValueError("form must be rows, columns or both, got %r" % (form,))
    if (out is not None and form == "columns") or (out_t is not None and form == "rows"):
        raise ValueError("form %r has no such output" % form)
    rows, cols, ld = _matrix(src, "src")
    device = src.device
    dt = dtype_code(src.dtype)
    a = t = None
    p = [None, None, None, None]
    if form != "columns":
        a = _target(out, rows, cols, device, stream, "out")
        p[0], p[1] = a.codes.data_ptr(), a.scales.data_ptr()
    if form != "rows":
        t = _target(out_t, cols, rows, device, stream, "out_t")
        p[2], p[3] = t.codes.data_ptr(), t.scales.data_ptr()
    _issue("fsdp_mx4_quantize", device, stream, src.data_ptr(), dt, rows, cols, ld, *p)
    return a if form == "rows" else t if form == "columns" else (a, t)


def _shards(shards):
    shards = list(shards)
    if not shards:
        raise ValueError("shards is empty")
    S = shards[0].cols
    for q, s in enumerate(shards):
        if not isinstance(s, Mx4) or s.rows != 1 or s.cols != S:
            raise ValueError("shards[%d] must be an Mx4 of one row and %d columns" % (q, S))
        _dev(s.codes, "shards[%d]" % q)
    return shards, len(shards), S, shards[0].device


def fsdp_mx4_gather(shards, full=None, dtype=torch.bfloat16, stream=None):
    """Gather the N ranks' quantised shards (Mx4 of one row) into the full flat
    buffer of `full`'s dtype (allocated in `dtype` if full is None)."""
    shards, world, S, device = _shards(shards)
    if full is None:
        with _on(stream):
            full = torch.empty(world * S, dtype=dtype, device=device)
    _dev(full, "full")
    if full.numel() != world * S:
        raise ValueError("full must hold world*shard = %d elements" % (world * S))
    _one_device(device, full, *(s.codes for s in shards))
    _issue("fsdp_mx4_gather", device, stream, ptr_array([s.codes.data_ptr() for s in shards]),
           ptr_array([s.scales.data_ptr() for s in shards]), world, S, dtype_code(full.dtype), full.data_ptr())
    return full


def fsdp_mx4_gather_packed(shards, full=None, stream=None):
    """Gather the N ranks' quantised shards as they are into one Mx4 of one row
    (the shard's size must be a multiple of 32)."""
    shards, world, S, device = _shards(shards)
    if S % BLOCK:
        raise ValueError("the shard's size %d is not a multiple of %d: the shards' blocks do not join" % (S, BLOCK))
    full = _target(full, 1, world * S, device, stream, "full")
    _one_device(device, full.codes, *(s.codes for s in shards))
    _issue("fsdp_mx4_gather_packed", device, stream, ptr_array([s.codes.data_ptr() for s in shards]),
           ptr_array([s.scales.data_ptr() for s in shards]), world, S, full.codes.data_ptr(), full.scales.data_ptr())
    return full


def fsdp_mx4_views(full, shapes):
    """Per-tensor matrices of a gathered packed unit, nothing copied: entry k is
    the Mx4 of tensor k (its last dimension the columns), or None where its
    offset or its last dimension is not a multiple of 32."""
    if not isinstance(full, Mx4) or full.rows != 1:
        raise ValueError("full must be an Mx4 of one row")
    out, off = [], 0
    codes, scales = full.codes.view(-1), full.scales.view(-1)
    for s in shapes:
        n = 1
        for x in s:
            n *= int(x)
        if off + n > full.cols:
            raise ValueError("the tensors hold more than the %d elements of the unit" % full.cols)
        cols = int(s[-1]) if len(s) else 1
        if n and off % BLOCK == 0 and cols % BLOCK == 0:
            out.append(Mx4(codes[off // 2:(off + n) // 2].view(n // cols, cols // 2),
                           scales[off // BLOCK:(off + n) // BLOCK].view(n // cols, cols // BLOCK), cols))
        else:
            out.append(None)
        off += n
    return out


def fsdp_mx4_matmul(a, b, out=None, dtype=torch.bfloat16, stream=None):
    """out[i, j] = sum_k a[i, k] b[j, k] of two Mx4 with equal columns; `out` may
    have strided rows and any alignment (a gradient's place in a flat buffer)."""
    for name, x in (("a", a), ("b", b)):
        if not isinstance(x, Mx4):
            raise TypeError("%s must be an Mx4" % name)
        if not x.codes.is_cuda:
            raise ValueError("%s must be on a device, got %s" % (name, x.device))
    if a.cols != b.cols:
        raise ValueError("a has %d columns, b %d" % (a.cols, b.cols))
    device = a.device
    out, ldo = _result(out, a.rows, b.rows, dtype, device, stream)
    _one_device(device, b.codes, out)
    _issue("fsdp_mx4_matmul", device, stream, a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(),
           b.scales.data_ptr(), a.rows, b.rows, a.cols, dtype_code(out.dtype), out.data_ptr(), ldo)
    return out


def _space(nbytes, device, stream):
    """(tensor that keeps it, address, bytes) of a call's workspace."""
    if nbytes <= 0:                              # none needed, or sizes that the call itself refuses
        return None, None, 0
    with _on(stream):
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), nbytes


def fsdp_mx4_linear(x, w, out=None, stream=None):
    """y = x W^T for x [tokens, in] and W an Mx4 [out, in]: x is quantised along
    its features on the way (for a few tokens within the one launch).  y has x's
    dtype unless `out` says otherwise, and no graph: where grad mode is on, an x
    that requires grad is refused."""
    if not isinstance(w, Mx4):
        raise TypeError("w must be an Mx4")
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != w.cols:
        raise ValueError("x must be a matrix of %d columns" % w.cols)
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("x requires grad, and y would carry none: call under torch.no_grad() or detach x, and take "
                         "the gradients from fsdp_mx4_linear_grads")
    m, k, ldx = _matrix(x, "x")
    device = x.device
    out, ldo = _result(out, m, w.rows, x.dtype, device, stream)
    _one_device(device, w.codes, out)
    keep, space, nbytes = _space(N.lib().fsdp_mx4_linear_workspace(m, k), device, stream)
    _issue("fsdp_mx4_linear", device, stream, x.data_ptr(), dtype_code(x.dtype), m, k, ldx, w.codes.data_ptr(),
           w.scales.data_ptr(), w.rows, dtype_code(out.dtype), out.data_ptr(), ldo, space, nbytes)
    return out


def fsdp_mx4_linear_grads(dy, x, wt, dx=None, dw=None, dw_dtype=None, stream=None):
    """Gradients of y = x W^T from dy [tokens, out] and x [tokens, in]:
    dx = dy W (dtype of x) and dw = dy^T x (dw_dtype, else the dtype of x), each
    the product of its operands quantised along the axis that it sums over.
    wt: W quantised along its columns, an Mx4 [in, out].  dx and dw may be given
    (dw: the weight's place in a flat gradient); dx=False or dw=False: not
    wanted, and None in its place."""
    if not isinstance(wt, Mx4):
        raise TypeError("wt must be an Mx4")
    for name, t, c in (("dy", dy, wt.cols), ("x", x, wt.rows)):
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] != c:
            raise ValueError("%s must be a matrix of %d columns" % (name, c))
    m, n, lddy = _matrix(dy, "dy")
    mx, k, ldx = _matrix(x, "x")
    if m != mx:
        raise ValueError("dy has %d rows, x %d" % (m, mx))
    device = dy.device
    want_dx, want_dw = dx is not False, dw is not False
    pdx = pdw = None
    lddx = lddw = cdx = cdw = 0
    _one_device(device, x, wt.codes)
    if want_dx:
        dx, lddx = _result(dx, m, k, x.dtype, device, stream)
        _one_device(device, dx)
        pdx, cdx = dx.data_ptr(), dtype_code(dx.dtype)
    if want_dw:
        dw, lddw = _result(dw, n, k, dw_dtype or x.dtype, device, stream)
        _one_device(device, dw)
        pdw, cdw = dw.data_ptr(), dtype_code(dw.dtype)
    keep, space, nbytes = _space(N.lib().fsdp_mx4_linear_grads_workspace(m, n, k, int(want_dx), int(want_dw)), device,
                                 stream)
    _issue("fsdp_mx4_linear_grads", device, stream, dy.data_ptr(), dtype_code(dy.dtype), lddy, x.data_ptr(),
           dtype_code(x.dtype), ldx, m, n, k, wt.codes.data_ptr(), wt.scales.data_ptr(), cdx, pdx, lddx, cdw, pdw,
           lddw, space, nbytes)
    return dx if want_dx else None, dw if want_dw else None
