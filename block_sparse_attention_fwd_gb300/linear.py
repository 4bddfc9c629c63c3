"""Operators of the linear layers around the attention, on torch tensors:
products of 8-bit codes with a scale for each block of 128, the layer norm, and
dropout whose mask is never stored.

As in ``ops.py``, each function checks its arguments, allocates its outputs and
makes one call of the C ABI in ``include/bl_attn.h`` on the current stream of
the tensors' device; all arithmetic runs in libbl_attn.so.  They stand outside
autograd; ``api.py`` builds the autograd modules from them.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from .ops import Act8, _empty_act8, _launch, _like, _rows, _tensor, _weight_dtype

_E4M3 = torch.float8_e4m3fn


# --- products in 8 bits ----------------------------------------------------------

class _Codes8:
    """e4m3 codes [rows, cols] (rows may be apart), their scales, and the type of
    the tensor that they stand for."""
    __slots__ = ("codes", "scales", "dtype", "stride")

    def __init__(self, codes, scales, dtype):
        if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
            raise TypeError("codes must be a CUDA tensor")
        if codes.dtype != _E4M3:
            raise TypeError(f"codes must be float8_e4m3fn, got {codes.dtype}")
        if dtype not in _lib.DTYPES:
            raise TypeError(f"the tensor was bf16, fp16 or fp32, got {dtype}")
        if codes.dim() != 2 or codes.shape[1] < 1:
            raise ValueError(f"codes are [rows, cols], got {tuple(codes.shape)}")
        rows, cols = codes.shape
        stride = codes.stride(0) if rows > 1 else cols
        if (cols > 1 and codes.stride(1) != 1) or stride < cols:
            raise ValueError(f"codes with strides {codes.stride()} are not rows apart")
        _tensor(scales, "scales", codes.device, torch.float32, self._scales_shape(rows, cols))
        self.codes, self.scales, self.dtype, self.stride = codes, scales, dtype, stride

    @property
    def shape(self):
        return self.codes.shape

    @property
    def nbytes(self):
        return self.codes.numel() + 4 * self.scales.numel()

    @classmethod
    def _empty(cls, rows, cols, dtype, device):
        """Rows 16-byte aligned, as the products want them."""
        a = cls.__new__(cls)
        a.stride = -(-cols // 16) * 16
        a.codes = torch.empty((rows, a.stride), dtype=_E4M3, device=device)
        if a.stride != cols:
            a.codes = a.codes[:, :cols]
        a.scales = torch.empty(cls._scales_shape(rows, cols), dtype=torch.float32, device=device)
        a.dtype = dtype
        return a

    def load(self):
        """The tensor that the codes stand for, in its type."""
        rows, cols = self.codes.shape
        x = torch.empty((rows, cols), dtype=self.dtype, device=self.codes.device)
        _launch("bl_tile8_load", x.device, rows, cols, _lib.DTYPES[self.dtype],
                self.codes.data_ptr(), self.stride, self.scales.data_ptr(), self._blocks,
                x.data_ptr())
        return x


class Weight8(_Codes8):
    """A weight [out, in] as e4m3 codes with one scale for every 128 x 128 elements:
    ``scales`` fp32 [ceil(out / 128), ceil(in / 128)].  ``dtype``: the type it was
    saved from."""
    __slots__ = ()
    _blocks = 1

    @staticmethod
    def _scales_shape(rows, cols):
        return (-(-rows // 128), -(-cols // 128))


class Cols8(_Codes8):
    """A tensor [rows, cols] as e4m3 codes with one scale for every 128 elements of a
    column: ``scales`` fp32 [ceil(rows / 128), cols]."""
    __slots__ = ()
    _blocks = 0

    @staticmethod
    def _scales_shape(rows, cols):
        return (-(-rows // 128), cols)


_TILE8_ARGS = struct.Struct("<6q7Qi4x")


def weight_save(w) -> Weight8:
    """A weight [out, in] (bf16, fp16 or fp32; a contiguous last dim) in e4m3 with one
    scale for every 128 x 128 elements.  Both ``matmul8`` and ``matmul8_gx`` read it."""
    rows, cols, stride = _rows(w, "w")
    if w.dim() != 2:
        raise ValueError(f"w is [out, in], got {tuple(w.shape)}")
    a = Weight8._empty(rows, cols, w.dtype, w.device)
    _launch("bl_tile8_save", w.device, _TILE8_ARGS.pack(
        rows, cols, stride, 0, 0, a.stride, w.data_ptr(), 0, 0, 0, 0, a.codes.data_ptr(),
        a.scales.data_ptr(), _lib.DTYPES[w.dtype]))
    return a


def act_save_both(x, rows=True, cols=True):
    """x [..., cols] (bf16, fp16 or fp32) in e4m3 in one reading: (its Act8 with groups
    of 128, bit for bit ``act_save(x, "e4m3", 128)``, and the Cols8 of x seen as
    [tokens, cols]); what is not asked for is None."""
    m, n, stride = _rows(x, "x")
    if not (rows or cols):
        raise ValueError("rows, cols or both")
    a = _empty_act8(x.shape, x.dtype, x.device, "e4m3", 128) if rows else None
    c = Cols8._empty(m, n, x.dtype, x.device) if cols else None
    _launch("bl_tile8_save", x.device, _TILE8_ARGS.pack(
        m, n, stride, n, c.stride if cols else 0, 0, x.data_ptr(),
        a.codes.data_ptr() if rows else 0, a.scales.data_ptr() if rows else 0,
        c.codes.data_ptr() if cols else 0, c.scales.data_ptr() if cols else 0, 0, 0,
        _lib.DTYPES[x.dtype]))
    return a, c


_MATMUL8_ARGS = struct.Struct("<3q2Qq2Qq3Q2i")


def _matmul8(form, tokens, n, k, a, a_stride, b, b_stride, shape, dtype):
    dev = a.codes.device
    if dtype not in _lib.DTYPES:
        raise TypeError(f"the result is bf16, fp16 or fp32, got {dtype}")
    if b.codes.device != dev:
        raise ValueError(f"codes on {dev} and {b.codes.device}")
    out = torch.empty(shape, dtype=dtype, device=dev)
    a_ptr, b_ptr = a.codes.data_ptr(), b.codes.data_ptr()
    args = [tokens, n, k, a_ptr, a.scales.data_ptr(), a_stride, b_ptr, b.scales.data_ptr(),
            b_stride, out.data_ptr(), 0, 0, form, _lib.DTYPES[dtype]]
    if (a_ptr | b_ptr | a_stride | b_stride) & 15:     # rows that the call copies first
        nbytes = _lib.load().bl_matmul8_workspace_bytes(_MATMUL8_ARGS.pack(*args))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        args[10:12] = ws.data_ptr(), nbytes
    _launch("bl_matmul8", dev, _MATMUL8_ARGS.pack(*args))
    return out


def _row_groups(a, name, cols):
    if not isinstance(a, Act8):
        raise TypeError(f"{name} must be an Act8")
    if a.codes.dtype != _E4M3 or a.group != 128:
        raise ValueError(f"{name} must be saved in e4m3 with groups of 128")
    if a.codes.shape[-1] != cols:
        raise ValueError(f"{name} has {a.codes.shape[-1]} columns, the weight {cols}")
    return a.codes.numel() // cols


def matmul8(x8, w8, dtype=None):
    """y = x w^T of x8, an Act8 [..., in] in e4m3 with groups of 128 (``act_save``,
    ``act_save_both``, ``rms_norm_fwd_8bit``, ``layer_norm_fwd_8bit``), and w8, the Weight8
    [out, in]: [..., out] in ``dtype`` (that x was saved from)."""
    if not isinstance(w8, Weight8):
        raise TypeError("w8 must be a Weight8")
    n, k = w8.codes.shape
    m = _row_groups(x8, "x8", k)
    return _matmul8(0, m, n, k, x8, k, w8, w8.stride, (*x8.codes.shape[:-1], n),
                    dtype or x8.dtype)


def matmul8_gx(g8, w8, dtype=None):
    """g_x = g_y w, the gradient of ``matmul8``'s x, of g8, the Act8 [..., out] of g_y
    in e4m3 with groups of 128, and w8 [out, in]: [..., in] in ``dtype`` (g8's)."""
    if not isinstance(w8, Weight8):
        raise TypeError("w8 must be a Weight8")
    n, k = w8.codes.shape
    m = _row_groups(g8, "g8", n)
    return _matmul8(1, m, n, k, g8, n, w8, w8.stride, (*g8.codes.shape[:-1], k),
                    dtype or g8.dtype)


def matmul8_gw(g8, x8, dtype=None):
    """g_w = g_y^T x, the gradient of ``matmul8``'s weight, of the Cols8 of g_y [tokens,
    out] and of x [tokens, in]: [out, in] in ``dtype`` (g8's)."""
    for a, name in ((g8, "g8"), (x8, "x8")):
        if not isinstance(a, Cols8):
            raise TypeError(f"{name} must be a Cols8")
    if g8.codes.shape[0] != x8.codes.shape[0]:
        raise ValueError(f"{g8.codes.shape[0]} and {x8.codes.shape[0]} tokens")
    m, n = g8.codes.shape
    k = x8.codes.shape[1]
    return _matmul8(2, m, n, k, g8, g8.stride, x8, x8.stride, (n, k), dtype or g8.dtype)


# --- layer norm --------------------------------------------------------------------

_LAYER_NORM_ARGS = struct.Struct("<4q9Qf2i4x")
_LAYER_NORM_BWD_ARGS = struct.Struct("<2q12Q2i")


def _affine_dtype(weight, bias, dtype, cols, device):
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight and bias of one type, got {weight.dtype} and {bias.dtype}")
    if bias is not None:
        if bias.dtype not in (dtype, torch.float32):
            raise TypeError(f"bias must be {dtype} or fp32, got {bias.dtype}")
        _tensor(bias, "bias", device, None, (cols,))
    if weight is None and bias is not None:
        return _lib.DTYPES[bias.dtype]
    return _weight_dtype(weight, dtype, cols, device)


def _layer_fwd(x, weight, bias, eps, residual, want_y, y8):
    rows, cols, stride = _rows(x, "x")
    if cols > _lib.NORM_MAX_COLS:
        raise ValueError(f"rows of {cols} elements: the norm takes up to {_lib.NORM_MAX_COLS}")
    dtype, device, shape = x.dtype, x.device, x.shape
    wtype = _affine_dtype(weight, bias, dtype, cols, device)
    h, r_ptr, h_ptr, r_stride = x, 0, 0, cols
    if residual is not None:
        if residual.dtype != dtype or residual.shape != shape or residual.device != device:
            raise ValueError("the residual must have x's type, shape and device, got "
                             f"{residual.dtype} {tuple(residual.shape)} on {residual.device}")
        r_stride = _rows(residual, "residual")[2]
        h = _like(x)
        r_ptr, h_ptr = residual.data_ptr(), h.data_ptr()
    y = _like(x) if want_y else None
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    rstd = torch.empty_like(mean)
    s8 = None if y8 is None else y8.struct()
    _launch("bl_layer_norm_fwd", device, _LAYER_NORM_ARGS.pack(
        rows, cols, stride, r_stride, x.data_ptr(), r_ptr,
        0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
        0 if y is None else y.data_ptr(), h_ptr, mean.data_ptr(), rstd.data_ptr(),
        0 if s8 is None else ctypes.addressof(s8), eps, _lib.DTYPES[dtype], wtype))
    return y, h, mean, rstd


def layer_norm_fwd(x, weight, bias, eps=1e-5, residual=None):
    """h = x + residual, m = mean(h), rstd = 1 / sqrt(mean((h - m)^2) + eps) over the
    last dim, y = (h - m) * rstd * weight + bias.  x (and residual): bf16, fp16 or fp32
    with a contiguous last dim of up to 16384; weight and bias: x's type or fp32, both
    the same, or None.  Returns (y, h, m, rstd); without a residual h is x itself."""
    return _layer_fwd(x, weight, bias, eps, residual, True, None)


def layer_norm_fwd_8bit(x, weight, bias, eps=1e-5, residual=None, fmt="e4m3", group=128,
                        with_y=False):
    """``layer_norm_fwd`` with y in 8 bits: returns (y8, h, m, rstd), or with ``with_y``
    (y, y8, h, m, rstd)."""
    y8 = _empty_act8(x.shape, x.dtype, x.device, fmt, group)
    y, h, mean, rstd = _layer_fwd(x, weight, bias, eps, residual, with_y, y8)
    return (y, y8, h, mean, rstd) if with_y else (y8, h, mean, rstd)


def layer_norm_bwd(g_y, h, mean, rstd, weight, g_h=None, need_g_w=True, need_g_b=True):
    """Gradients of ``layer_norm_fwd``: (g_x, g_w, g_b).  ``h`` is the forward's h or
    its Act8; ``g_h``, the gradient that reaches h along the residual stream, is added
    to g_x, which is the residual's gradient too.  g_w and g_b have the weight's type
    (fp32 without a weight); None when not needed."""
    rows, cols, _ = _rows(g_y, "g_y")
    if not g_y.is_contiguous():
        raise ValueError("g_y must be contiguous")
    if cols > _lib.NORM_MAX_COLS:
        raise ValueError(f"rows of {cols} elements: the norm takes up to {_lib.NORM_MAX_COLS}")
    dev, dtype = g_y.device, g_y.dtype
    h_ptr, s8 = 0, None
    if isinstance(h, Act8):
        _tensor(h.codes, "h", dev, None, g_y.shape)
        if h.dtype != dtype:
            raise TypeError(f"h was saved from {h.dtype}, g_y is {dtype}")
        s8 = h.struct()
    else:
        _tensor(h, "h", dev, dtype, g_y.shape)
        h_ptr = h.data_ptr()
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _tensor(t, name, dev, torch.float32)
        if t.numel() != rows:
            raise ValueError(f"{name} has {t.numel()} elements for {rows} rows")
    if g_h is not None:
        _tensor(g_h, "g_h", dev, dtype, g_y.shape)
    wtype = 2 if weight is None else _weight_dtype(weight, dtype, cols, dev)
    g_type = torch.float32 if weight is None else weight.dtype
    g_x = torch.empty_like(g_y)
    g_w = torch.empty(cols, dtype=g_type, device=dev) if need_g_w else None
    g_b = torch.empty(cols, dtype=g_type, device=dev) if need_g_b else None
    ws_ptr = nbytes = 0
    if need_g_w or need_g_b:
        nbytes = _lib.load().bl_layer_norm_bwd_workspace_bytes(rows, cols)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws_ptr = ws.data_ptr()
    _launch("bl_layer_norm_bwd", dev, _LAYER_NORM_BWD_ARGS.pack(
        rows, cols, g_y.data_ptr(), h_ptr, 0 if s8 is None else ctypes.addressof(s8),
        mean.data_ptr(), rstd.data_ptr(), 0 if weight is None else weight.data_ptr(),
        0 if g_h is None else g_h.data_ptr(), g_x.data_ptr(), 0 if g_w is None else g_w.data_ptr(),
        0 if g_b is None else g_b.data_ptr(), ws_ptr, nbytes, _lib.DTYPES[dtype], wtype))
    return g_x, g_w, g_b


# --- dropout -----------------------------------------------------------------------

def _state(state, device=None):
    _tensor(state, "state", device, torch.int64, (2,))


def dropout(x, p, state, residual=None):
    """y = x / (1 - p) where an element is kept, else 0, plus ``residual``.  x (and
    residual): bf16, fp16 or fp32 with a contiguous last dim.  Element i of x (in
    row-major order, whatever the strides) is kept iff word i % 4 of Philox4x32-10 of
    the counter (i / 4, offset) and the key `seed` is at least round(p * 2^32);
    ``state`` is the int64 CUDA tensor (seed, offset), read when the kernel runs.  The
    gradient is the same call on g_y: ``dropout(g_y, p, state)``."""
    rows, cols, stride = _rows(x, "x")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must lie in [0, 1], got {p}")
    _state(state, x.device)
    r_ptr, r_stride = None, cols
    if residual is not None:
        if residual.dtype != x.dtype or residual.shape != x.shape or residual.device != x.device:
            raise ValueError("the residual must have x's type, shape and device, got "
                             f"{residual.dtype} {tuple(residual.shape)} on {residual.device}")
        r_stride = _rows(residual, "residual")[2]
        r_ptr = residual.data_ptr()
    y = _like(x)
    _launch("bl_dropout", x.device, rows, cols, _lib.DTYPES[x.dtype], x.data_ptr(), stride, r_ptr,
            r_stride, float(p), state.data_ptr(), y.data_ptr())
    return y


def dropout_next(state):
    """The state of this call, a copy of ``state``, whose offset then goes one on: in
    stream order, so that a captured graph draws anew with every replay."""
    _state(state)
    used = torch.empty_like(state)
    _launch("bl_dropout_next", state.device, state.data_ptr(), used.data_ptr())
    if not state.is_inference():           # what autograd holds of it is stale now
        torch.autograd.graph.increment_version(state)
    return used
