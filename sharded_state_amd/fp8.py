"""8-bit blocks: the compute copy at 129/128 byte an element, its all-gather,
and products of matrices kept that way.

Blocks of 128 elements share a power of two; an element is an e4m3 number
(include/fsdp_shard.h has the format to the bit).

    mine = ss.fsdp_fp8_quantize(master)                    # this rank's shard
    full = ss.fsdp_fp8_gather(shards, full)                # N shards -> the 16-bit full buffer
    packed = ss.fsdp_fp8_gather_packed(shards)             # N shards -> one packed unit
    w = ss.fsdp_fp8_views(packed, shapes)[k]               # a weight of it, nothing copied
    y = ss.fsdp_fp8_linear(x, w)                           # x quantised on the way, y = x W^T

A product needs its blocks along the summed axis.  The forward sums over the
input features, the gradient of x over the output features and the gradient of
W over the tokens, so ``fsdp_fp8_linear_grads`` quantises dy and x along the
axes that it sums over and takes W quantised along its columns.  A weight with
one scale for each 128 x 128 elements holds the same values in both directions:

    w, wt = ss.fsdp_fp8_quantize(w16, form="both", tile=True)

Quantisation itself is passed through unchanged by the gradients.
"""
import torch

from . import _native as N
from ._native import ptr_array
from .api import _changed, _dev, _issue, _no_tangents, _on, dtype_code
from .mx4 import _matrix, _one_device, _result, _space

BLOCK = 128


def _blocks(cols):
    return -(-cols // BLOCK)


class Fp8:
    """A matrix of `rows` x `cols` in 8-bit blocks along its rows.

    codes   uint8 [rows, ceil(cols / 128) * 128], contiguous, 16-byte aligned
    scales  uint8 [rows, ceil(cols / 128)], contiguous; with `tile`, one for each
            128 x 128 elements, [ceil(rows / 128), ceil(cols / 128)]"""

    __slots__ = ("_codes", "_scales", "_both", "rows", "cols", "tile", "device")

    def __init__(self, codes, scales, cols, tile=False):
        nb = _blocks(cols)
        for name, t, w in (("codes", codes, nb * BLOCK), ("scales", scales, nb)):
            if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[1] != w or not t.is_contiguous():
                raise ValueError("%s must be a contiguous uint8 matrix of %d columns for cols = %d" % (name, w, cols))
        rows = codes.shape[0]
        if scales.shape[0] != (_blocks(rows) if tile else rows):
            raise ValueError("codes has %d rows, scales %d%s" % (rows, scales.shape[0], " of tiles" if tile else ""))
        if codes.device != scales.device:
            raise ValueError("codes is on %s, scales on %s" % (codes.device, scales.device))
        if codes.data_ptr() % 16:
            raise ValueError("codes must be 16-byte aligned")
        self._codes, self._scales, self._both = codes, scales, None
        self.rows, self.cols, self.tile, self.device = rows, int(cols), bool(tile), codes.device

    @classmethod
    def empty(cls, rows, cols, device="cuda", tile=False):
        """Not filled: one allocation, the scales behind the codes."""
        self = object.__new__(cls)               # what is allocated here needs no check
        nb = _blocks(cols)
        n = rows * nb * BLOCK + (_blocks(rows) if tile else rows) * nb
        self._codes, self._scales, self._both = None, None, torch.empty(n, dtype=torch.uint8, device=device)
        self.rows, self.cols, self.tile, self.device = rows, cols, bool(tile), self._both.device
        return self

    def _views(self):
        both = self._both
        if both is None:                         # made meanwhile, by another thread
            return
        nb = _blocks(self.cols)
        behind = self.rows * nb * BLOCK
        self._scales = both[behind:].view(_blocks(self.rows) if self.tile else self.rows, nb)
        self._codes = both[:behind].view(self.rows, nb * BLOCK)
        self._both = None                        # from here on the views are the matrix, copied or pickled as such

    @property
    def codes(self):
        if self._codes is None:
            self._views()
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._views()
        return self._scales

    def _ptrs(self):
        """The addresses of codes and scales."""
        both = self._both
        if both is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        at = both.data_ptr()
        return at, at + self.rows * _blocks(self.cols) * BLOCK

    @property
    def shape(self):
        return (self.rows, self.cols)

    def __repr__(self):
        return "Fp8(%d x %d, %s%s)" % (self.rows, self.cols, self.device, ", in tiles" if self.tile else "")


def _target(out, rows, cols, tile, device, stream, name):
    if out is None:
        if stream is None:
            return Fp8.empty(rows, cols, device, tile)
        with _on(stream):
            return Fp8.empty(rows, cols, device, tile)
    if not isinstance(out, Fp8):
        raise TypeError("%s must be an Fp8" % name)
    if out.shape != (rows, cols) or out.device != device or out.tile != tile:
        raise ValueError("%s must be %d x %d %son %s, got %r" % (name, rows, cols, "in tiles " if tile else "", device, out))
    return out


def _operand(t, name):
    if not isinstance(t, Fp8):
        raise TypeError("%s must be an Fp8" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a device, got %s" % (name, t.device))
    return t


def fsdp_fp8_quantize(src, out=None, out_t=None, form="rows", tile=False, stream=None):
    """A flat shard (1-D: one row) or a matrix (2-D, its rows may be strided) of
    float32, float16 or bfloat16 in 8-bit blocks.  form "rows": blocks along the
    rows, as Fp8 of src's shape; "columns": blocks along the columns, as Fp8 of
    the transpose's shape; "both": the two of them.  tile: one scale for each
    128 x 128 elements; both forms then hold the same values."""
    if form not in ("rows", "columns", "both"):
        raise ValueError("form must be rows, columns or both, got %r" % (form,))
    if (out is not None and form == "columns") or (out_t is not None and form == "rows"):
        raise ValueError("form %r has no such output" % form)
    rows, cols, ld = _matrix(src, "src")
    device, tile = src.device, bool(tile)
    dt = dtype_code(src.dtype)
    a = t = None
    p = [None, None, None, None]
    if form != "columns":
        a = _target(out, rows, cols, tile, device, stream, "out")
        p[0], p[1] = a._ptrs()
    if form != "rows":
        t = _target(out_t, cols, rows, tile, device, stream, "out_t")
        p[2], p[3] = t._ptrs()
    _issue("fsdp_fp8_quantize", device, stream, src.data_ptr(), dt, rows, cols, ld, int(tile), *p)
    return a if form == "rows" else t if form == "columns" else (a, t)


def _shards(shards):
    shards = list(shards)
    if not shards:
        raise ValueError("shards is empty")
    S = shards[0].cols if isinstance(shards[0], Fp8) else 0
    for q, s in enumerate(shards):
        if not isinstance(s, Fp8) or s.rows != 1 or s.cols != S:
            raise ValueError("shards[%d] must be an Fp8 of one row and %d columns" % (q, S))
        _operand(s, "shards[%d]" % q)
    return shards, len(shards), S, shards[0].device


def fsdp_fp8_gather(shards, full=None, dtype=torch.bfloat16, stream=None):
    """Gather the N ranks' quantised shards (Fp8 of one row) into the full flat
    buffer of `full`'s dtype (allocated in `dtype` if full is None)."""
    shards, world, S, device = _shards(shards)
    if full is None:
        with _on(stream):
            full = torch.empty(world * S, dtype=dtype, device=device)
    _dev(full, "full")
    if full.numel() != world * S:
        raise ValueError("full must hold world*shard = %d elements" % (world * S))
    _one_device(device, full, *shards)
    codes, scales = zip(*(s._ptrs() for s in shards))
    _issue("fsdp_fp8_gather", device, stream, ptr_array(codes), ptr_array(scales), world, S, dtype_code(full.dtype), full.data_ptr())
    return full


def fsdp_fp8_gather_packed(shards, full=None, stream=None):
    """Gather the N ranks' quantised shards as they are into one Fp8 of one row
    (the shard's size must be a multiple of 128)."""
    shards, world, S, device = _shards(shards)
    if S % BLOCK:
        raise ValueError("the shard's size %d is not a multiple of %d: the shards' blocks do not join" % (S, BLOCK))
    full = _target(full, 1, world * S, False, device, stream, "full")
    _one_device(device, *shards)
    codes, scales = zip(*(s._ptrs() for s in shards))
    _issue("fsdp_fp8_gather_packed", device, stream, ptr_array(codes), ptr_array(scales), world, S, *full._ptrs())
    return full


def fsdp_fp8_views(full, shapes):
    """Per-tensor matrices of a gathered packed unit, nothing copied: entry k is
    the Fp8 of tensor k (its last dimension the columns), or None where its
    offset or its last dimension is not a multiple of 128."""
    if not isinstance(full, Fp8) or full.rows != 1 or full.tile:
        raise ValueError("full must be an Fp8 of one row, not in tiles")
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
            out.append(Fp8(codes[off:off + n].view(n // cols, cols),
                           scales[off // BLOCK:(off + n) // BLOCK].view(n // cols, cols // BLOCK), cols))
        else:
            out.append(None)
        off += n
    return out


def fsdp_fp8_matmul(a, b, out=None, dtype=torch.bfloat16, stream=None):
    """out[i, j] = sum_k a[i, k] b[j, k] of two Fp8 with equal columns; `out` may
    have strided rows and any alignment (a gradient's place in a flat buffer)."""
    _operand(a, "a")
    _operand(b, "b")
    if a.cols != b.cols:
        raise ValueError("a has %d columns, b %d" % (a.cols, b.cols))
    m, n, k, device = a.rows, b.rows, a.cols, a.device
    given = out
    out, ldo = _result(out, m, n, dtype, device, stream)
    _one_device(device, b, out)
    keep, space, nbytes = _space(N.lib().fsdp_fp8_matmul_workspace(m, n, k), device, stream)
    _issue("fsdp_fp8_matmul", device, stream, *a._ptrs(), int(a.tile), *b._ptrs(),
           int(b.tile), m, n, k, dtype_code(out.dtype), out.data_ptr(), ldo, space, nbytes)
    _changed(given)
    return out


def fsdp_fp8_linear(x, w, out=None, dtype=None, stream=None):
    """y = x W^T for x [tokens, in] and W an Fp8 [out, in].  x is a tensor, which
    is quantised along its features on the way, or an Fp8 (what
    ``fsdp_rms_norm_fp8`` gives).  y has `out`'s dtype, else `dtype`, else x's
    (bfloat16 for an Fp8), and no graph: where grad mode is on, an x that requires
    grad is refused, and so is one with a forward-mode tangent."""
    _operand(w, "w")
    if isinstance(x, Fp8):
        if x.cols != w.cols:
            raise ValueError("x must be a matrix of %d columns" % w.cols)
        return fsdp_fp8_matmul(x, w, out, dtype or torch.bfloat16, stream)
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != w.cols:
        raise ValueError("x must be a matrix of %d columns" % w.cols)
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("x requires grad, and y would carry none: call under torch.no_grad() or detach x, and take "
                         "the gradients from fsdp_fp8_linear_grads")
    _no_tangents(x)
    m, k, ldx = _matrix(x, "x")
    n, device = w.rows, x.device
    given = out
    out, ldo = _result(out, m, n, dtype or x.dtype, device, stream)
    _one_device(device, w, out)
    keep, space, nbytes = _space(N.lib().fsdp_fp8_linear_workspace(m, n, k), device, stream)
    _issue("fsdp_fp8_linear", device, stream, x.data_ptr(), dtype_code(x.dtype), m, k, ldx, *w._ptrs(),
           int(w.tile), n, dtype_code(out.dtype), out.data_ptr(), ldo, space, nbytes)
    _changed(given)
    return out


def fsdp_fp8_linear_grads(dy, x, wt, dx=None, dw=None, dw_dtype=None, stream=None):
    """Gradients of y = x W^T from dy [tokens, out] and x [tokens, in]:
    dx = dy W (dtype of x) and dw = dy^T x (dw_dtype, else the dtype of x), each
    the product of its operands quantised along the axis that it sums over.
    wt: W quantised along its columns, an Fp8 [in, out].  dx and dw may be given
    (dw: the weight's place in a flat gradient); dx=False or dw=False: not
    wanted, and None in its place."""
    _operand(wt, "wt")
    for name, t, c in (("dy", dy, wt.cols), ("x", x, wt.rows)):
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] != c:
            raise ValueError("%s must be a matrix of %d columns" % (name, c))
    _no_tangents(dy, x)
    m, n, lddy = _matrix(dy, "dy")
    mx, k, ldx = _matrix(x, "x")
    if m != mx:
        raise ValueError("dy has %d rows, x %d" % (m, mx))
    device = dy.device
    want_dx, want_dw = dx is not False, dw is not False
    given = dx, dw
    pdx = pdw = None
    lddx = lddw = cdx = cdw = 0
    _one_device(device, x, wt)
    if want_dx:
        dx, lddx = _result(dx, m, k, x.dtype, device, stream)
        _one_device(device, dx)
        pdx, cdx = dx.data_ptr(), dtype_code(dx.dtype)
    if want_dw:
        dw, lddw = _result(dw, n, k, dw_dtype or x.dtype, device, stream)
        _one_device(device, dw)
        pdw, cdw = dw.data_ptr(), dtype_code(dw.dtype)
    keep, space, nbytes = _space(N.lib().fsdp_fp8_linear_grads_workspace(m, n, k, int(want_dx), int(want_dw)), device,
                                 stream)
    _issue("fsdp_fp8_linear_grads", device, stream, dy.data_ptr(), dtype_code(dy.dtype), lddy, x.data_ptr(),
           dtype_code(x.dtype), ldx, m, n, k, *wt._ptrs(), int(wt.tile), cdx, pdx, lddx,
           cdw, pdw, lddw, space, nbytes)
    _changed(*given)
    return dx if want_dx else None, dw if want_dw else None
