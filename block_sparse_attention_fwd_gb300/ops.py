"""Operators around the attention, on torch tensors: rotary positions with
several axes, the root-mean-square norm with the residual's addition, and
activations held in 8 bits until the backward.

Each function checks its arguments, allocates its outputs and makes one call
of the C ABI in ``include/bl_attn.h`` on the current stream of the tensors'
device; all arithmetic runs in libbl_attn.so.  They stand outside autograd:
their outputs carry no gradients.  ``api.py`` builds the autograd modules from
them.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

import torch

from . import _lib


def _launch(name, device, *args):
    """Calls a C entry point with the current stream of `device`."""
    index = device.index
    fn = getattr(_lib.load(), name)
    if _current_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, _raw_stream(index))
    if code != 0:
        raise _lib.BLError(name, code)


# The public calls build objects around these two numbers, which takes longer
# than a small launch; they are the fallback.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _tensor(t, name, device=None, dtype=None, shape=None):
    """Checks a contiguous CUDA tensor argument."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def row_stride(t):
    """Stride of the rows of the last dim, if they are equally spaced and each
    is contiguous; None where the tensor is no such run of rows."""
    cols = t.shape[-1]
    if t.is_contiguous():
        return cols
    if cols > 1 and t.stride(-1) != 1:
        return None
    stride, run = None, 1                   # run: rows covered by the dims behind
    for size, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * run:
            return None
        run *= size
    if stride is None:
        return cols
    return stride if stride >= cols else None


def _rows(t, name):
    """(rows, cols, row stride) of a tensor argument."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _lib.DTYPES:
        raise TypeError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    shape = t.shape
    cols = shape[-1] if shape else 0
    if cols < 1:
        raise ValueError(f"{name} needs a last dim of at least one element")
    if t.is_contiguous():
        return t.numel() // cols, cols, cols
    stride = row_stride(t)
    if stride is None:
        raise ValueError(f"{name} with strides {tuple(t.stride())} is not a run of rows")
    return t.numel() // cols, cols, stride


# --- activations in 8 bits -----------------------------------------------------

class Act8:
    """A tensor held in 8 bits: ``codes`` (int8 or float8_e4m3fn, the tensor's
    shape), ``scales`` (fp32, one for every ``group`` = 32, 64 or 128 elements
    of a row of the last dim, or one a row with ``group`` = 0) and ``dtype``,
    the type it was saved from and is loaded in."""
    __slots__ = ("codes", "scales", "group", "dtype")

    def __init__(self, codes, scales, group, dtype):
        if codes.dtype not in _lib.FORMATS8:
            raise TypeError(f"codes must be int8 or float8_e4m3fn, got {codes.dtype}")
        if group not in (0, 32, 64, 128):
            raise ValueError(f"group must be 0, 32, 64 or 128, got {group}")
        if dtype not in _lib.DTYPES:
            raise TypeError(f"an activation is bf16, fp16 or fp32, got {dtype}")
        _tensor(codes, "codes")
        _tensor(scales, "scales", codes.device, torch.float32)
        shape = codes.shape
        cols = shape[-1] if shape else 0
        if cols < 1:
            raise ValueError("codes need a last dim of at least one element")
        want = codes.numel() // cols * _groups(cols, group)
        if scales.numel() != want:
            raise ValueError(f"{scales.numel()} scales for {want} groups")
        self.codes, self.scales, self.group, self.dtype = codes, scales, group, dtype

    @property
    def shape(self):
        return self.codes.shape

    @property
    def nbytes(self):
        return self.codes.numel() + 4 * self.scales.numel()

    def struct(self):
        return _lib.Act8Struct(self.codes.data_ptr(), self.scales.data_ptr(),
                               _lib.FORMATS8[self.codes.dtype], self.group)


_FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _groups(cols, group):
    return -(-cols // group) if group else 1


def _empty_act8(shape, dtype, device, fmt, group):
    if fmt not in _FORMATS:
        raise ValueError(f"format must be one of {tuple(_FORMATS)}, got {fmt!r}")
    if group not in (0, 32, 64, 128):
        raise ValueError(f"group must be 0, 32, 64 or 128, got {group}")
    a = Act8.__new__(Act8)
    a.codes = torch.empty(shape, dtype=_FORMATS[fmt], device=device)
    a.scales = torch.empty((*shape[:-1], _groups(shape[-1], group)), dtype=torch.float32,
                           device=device)
    a.group, a.dtype = group, dtype
    return a


def act_save(x, fmt="int8", group=0) -> Act8:
    """x (bf16, fp16 or fp32; a contiguous last dim) in 8 bits, ``fmt`` "int8" or
    "e4m3", with one scale for every ``group`` elements of a row (0: one a row)."""
    rows, cols, stride = _rows(x, "x")
    a = _empty_act8(x.shape, x.dtype, x.device, fmt, group)
    _launch("bl_act_save", x.device, rows, cols, _lib.DTYPES[x.dtype], x.data_ptr(), stride,
            ctypes.byref(a.struct()))
    return a


def act_load(a):
    """The tensor an Act8 (or a Weight8 or Cols8) stands for, in the type it was saved
    from."""
    if not isinstance(a, Act8):
        return a.load()
    x = torch.empty(a.codes.shape, dtype=a.dtype, device=a.codes.device)
    cols = x.shape[-1]
    _launch("bl_act_load", x.device, x.numel() // cols, cols, _lib.DTYPES[a.dtype],
            ctypes.byref(a.struct()), x.data_ptr())
    return x


def attn_bwd_act8(shape, q8, k8, v8, o, g_o, lse, scale, lists=None, workspace=None):
    """The attention's backward (``attn_bwd``) from an 8-bit checkpoint: q8, k8
    and v8 are Act8 of [B, n, heads, d] with one scale a (token, head)
    (``act_save(q)``); ``o`` is the bf16 output or its Act8.  Returns (g_q, g_k,
    g_v).  ``workspace``: uint8, at least ``attn_bwd_act8_workspace_bytes(shape)``
    (allocated when None); ``bwd_check_status`` reads it like attn_bwd's."""
    B, n, H, Hk, d = shape.B, shape.n, shape.H, shape.Hk, shape.d
    dev = g_o.device
    for a, name, heads in ((q8, "q8", H), (k8, "k8", Hk), (v8, "v8", Hk)) + \
            (((o, "o", H),) if isinstance(o, Act8) else ()):
        if not isinstance(a, Act8):
            raise TypeError(f"{name} must be an Act8")
        _tensor(a.codes, name, dev, q8.codes.dtype, (B, n, heads, d))
        if a.group or a.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be saved from bf16 with one scale a row (group 0)")
    if not isinstance(o, Act8):
        _tensor(o, "o", dev, torch.bfloat16, (B, n, H, d))
    _tensor(g_o, "g_o", dev, torch.bfloat16, (B, n, H, d))
    _tensor(lse, "lse", dev, torch.float32, (B, H, n))
    ls = None
    if lists is not None:
        T_r, T_c = _lib.tiles(shape)
        _tensor(lists["q_idx"], "q_idx", dev, torch.int32, (B, H, T_c, T_r))
        _tensor(lists["q_cnt"], "q_cnt", dev, torch.int32, (B, H, T_c))
        ls = ctypes.byref(_lib._lists_struct(lists))
    if workspace is None:
        workspace = torch.empty(attn_bwd_act8_workspace_bytes(shape), dtype=torch.uint8, device=dev)
    else:
        _tensor(workspace, "workspace", dev, torch.uint8)
    g_q = torch.empty_like(g_o)
    g_k, g_v = (torch.empty((B, n, Hk, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    o8 = ctypes.byref(o.struct()) if isinstance(o, Act8) else None
    _launch("bl_attn_bwd_act8", dev, ctypes.byref(shape), ctypes.byref(q8.struct()),
            ctypes.byref(k8.struct()), ctypes.byref(v8.struct()),
            None if o8 is not None else o.data_ptr(), o8, g_o.data_ptr(), lse.data_ptr(),
            float(scale), ls, g_q.data_ptr(), g_k.data_ptr(), g_v.data_ptr(),
            workspace.data_ptr(), workspace.numel())
    return g_q, g_k, g_v


def attn_bwd_act8_workspace_bytes(shape) -> int:
    return int(_lib.load().bl_attn_bwd_act8_workspace_bytes(ctypes.byref(shape)))


# --- root-mean-square norm -------------------------------------------------------

def _weight_dtype(weight, dtype, cols, device):
    if weight is None:
        return _lib.DTYPES[dtype]
    if weight.dtype != dtype and weight.dtype != torch.float32:
        raise TypeError(f"weight must be {dtype} or fp32, got {weight.dtype}")
    _tensor(weight, "weight", device, None, (cols,))
    return _lib.DTYPES[weight.dtype]


def _norm_fwd(x, weight, eps, residual, want_y, y8):
    rows, cols, stride = _rows(x, "x")
    if cols > _lib.NORM_MAX_COLS:
        raise ValueError(f"rows of {cols} elements: the norm takes up to {_lib.NORM_MAX_COLS}")
    dtype, device, shape = x.dtype, x.device, x.shape
    wtype = _weight_dtype(weight, dtype, cols, device)
    h = r_ptr = h_ptr = None
    r_stride = cols
    if residual is not None:
        if residual.dtype != dtype or residual.shape != shape or residual.device != device:
            raise ValueError("the residual must have x's type, shape and device, got "
                             f"{residual.dtype} {tuple(residual.shape)} on {residual.device}")
        r_stride = _rows(residual, "residual")[2]
        h = _like(x)
        r_ptr, h_ptr = residual.data_ptr(), h.data_ptr()
    y = _like(x) if want_y else None
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    _launch("bl_rms_norm_fwd", device, rows, cols, _lib.DTYPES[dtype], x.data_ptr(), stride,
            r_ptr, r_stride, None if weight is None else weight.data_ptr(), wtype, eps,
            None if y is None else y.data_ptr(), h_ptr, rstd.data_ptr(),
            None if y8 is None else ctypes.byref(y8.struct()))
    return y, x if h is None else h, rstd


def _like(x):
    """An empty contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else \
        torch.empty(x.shape, dtype=x.dtype, device=x.device)


def rms_norm_fwd(x, weight, eps=1e-6, residual=None):
    """h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps) over the last dim,
    y = h * rstd * weight.  x (and residual): bf16, fp16 or fp32 with a
    contiguous last dim of up to 16384; weight: x's type or fp32, or None.
    Returns (y, h, rstd); without a residual h is x itself."""
    return _norm_fwd(x, weight, eps, residual, True, None)


def rms_norm_fwd_8bit(x, weight, eps=1e-6, residual=None, fmt="e4m3", group=128, with_y=False):
    """``rms_norm_fwd`` with y in 8 bits: returns (y8, h, rstd), or with ``with_y``
    (y, y8, h, rstd): y for the forward's product, y8 as its checkpoint."""
    y8 = _empty_act8(x.shape, x.dtype, x.device, fmt, group)
    y, h, rstd = _norm_fwd(x, weight, eps, residual, with_y, y8)
    return (y, y8, h, rstd) if with_y else (y8, h, rstd)


def rms_norm_bwd(g_y, h, rstd, weight, g_h=None, need_g_w=True):
    """Gradients of ``rms_norm_fwd``: (g_x, g_w).  ``h`` is the forward's h or
    its Act8; ``g_h``, the gradient that reaches h along the residual stream,
    is added to g_x, which is the residual's gradient too.  g_w has the
    weight's type (fp32 without a weight: the gradient of a weight of ones);
    None when not needed."""
    rows, cols, _ = _rows(g_y, "g_y")
    if not g_y.is_contiguous():
        raise ValueError("g_y must be contiguous")
    if cols > _lib.NORM_MAX_COLS:
        raise ValueError(f"rows of {cols} elements: the norm takes up to {_lib.NORM_MAX_COLS}")
    dev, dtype = g_y.device, g_y.dtype
    h8 = None
    if isinstance(h, Act8):
        _tensor(h.codes, "h", dev, None, g_y.shape)
        if h.dtype != dtype:
            raise TypeError(f"h was saved from {h.dtype}, g_y is {dtype}")
        h8 = ctypes.byref(h.struct())
    else:
        _tensor(h, "h", dev, dtype, g_y.shape)
    _tensor(rstd, "rstd", dev, torch.float32)
    if rstd.numel() != rows:
        raise ValueError(f"rstd has {rstd.numel()} elements for {rows} rows")
    if g_h is not None:
        _tensor(g_h, "g_h", dev, dtype, g_y.shape)
    wtype = 2 if weight is None else _weight_dtype(weight, dtype, cols, dev)
    g_x = torch.empty_like(g_y)
    g_w, ws, nbytes = None, None, 0
    if need_g_w:
        g_w = torch.empty(cols, dtype=torch.float32 if weight is None else weight.dtype, device=dev)
        nbytes = _lib.load().bl_rms_norm_bwd_workspace_bytes(rows, cols)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _launch("bl_rms_norm_bwd", dev, rows, cols, _lib.DTYPES[dtype], g_y.data_ptr(),
            None if h8 is not None else h.data_ptr(), h8, rstd.data_ptr(),
            None if weight is None else weight.data_ptr(), wtype,
            None if g_h is None else g_h.data_ptr(), g_x.data_ptr(),
            None if g_w is None else g_w.data_ptr(), None if ws is None else ws.data_ptr(), nbytes)
    return g_x, g_w


# --- rotary positions ------------------------------------------------------------

# 2 pi * 10^50, for frequencies in turns without an fp64 rounding
_TWO_PI_E50 = 628318530717958647692528676655900576839433879875021


@functools.lru_cache(maxsize=64)
def _fixed_point_freqs(freqs):
    """round(f / (2 pi) * 2^64) modulo 2^64 of each fp64 frequency, as int64."""
    out = []
    for f in freqs:
        num, den = float(f).as_integer_ratio()
        turns = (2 * (num << 64) * 10 ** 50 + den * _TWO_PI_E50) // (2 * den * _TWO_PI_E50)
        turns %= 1 << 64
        out.append(turns - (1 << 64) if turns >> 63 else turns)
    return out


class RopePlan:
    """Which pairs of a head turn with which axis and how fast; made once for a
    model and device.

    ``sections`` deals the first ``sum(sections)`` pairs of a head of
    ``head_dim`` dimensions to the axes in order (one section: the ordinary
    rotation; (22, 21, 21) for time, height and width at head_dim 128); the
    dimensions behind pass through.  ``layout`` "interleaved" pairs the
    dimensions (2p, 2p + 1), "half" (p, p + pairs).  Pair j of a section of m
    turns by theta^(-j / m) radians a position; with ``shared`` the pairs count
    through all sections (theta^(-p / pairs)); ``freqs`` gives every pair's
    frequency instead."""

    def __init__(self, head_dim, sections, theta=10000.0, layout="half", shared=False, freqs=None,
                 device="cuda"):
        sections = tuple(int(m) for m in sections)
        if not 1 <= len(sections) <= 4 or min(sections) < 1:
            raise ValueError(f"one to four sections of at least one pair, got {sections}")
        pairs = sum(sections)
        if not 2 <= head_dim <= 65536 or pairs > head_dim // 2:
            raise ValueError(f"{pairs} pairs do not fit a head of {head_dim} dimensions")
        if layout not in ("half", "interleaved"):
            raise ValueError(f'layout must be "half" or "interleaved", got {layout!r}')
        if freqs is None:
            if not (math.isfinite(theta) and theta > 0):
                raise ValueError(f"theta must be positive, got {theta}")
            if shared:
                freqs = [theta ** (-p / pairs) for p in range(pairs)]
            else:
                freqs = [theta ** (-j / m) for m in sections for j in range(m)]
        freqs = tuple(float(f) for f in freqs)
        if len(freqs) != pairs or not all(math.isfinite(f) for f in freqs):
            raise ValueError(f"{pairs} finite frequencies are needed, got {len(freqs)}")
        self.head_dim, self.sections, self.layout, self.pairs = head_dim, sections, layout, pairs
        self.freqs = freqs
        self.padded_sections = sections + (0,) * (4 - len(sections))
        self.fixed = torch.tensor(_fixed_point_freqs(freqs), dtype=torch.int64, device=device)


def _rope_strides(t, name, dtype, B, n, d):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape[:2] != (B, n) or t.shape[-1] != d:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({B}, {n}, heads, {d})")
    st = t.stride()
    if st[3] != 1:
        raise ValueError(f"{name} needs a contiguous last dim")
    return st[:3]


def rope(q, k, positions, plan, inverse=False, inplace=False):
    """Turns q [B, n, H, d] and k [B, n, Hk, d] (bf16, fp16 or fp32; views with a
    contiguous last dim; k may be None) by their positions, in one launch:
    ``positions`` is int32 [B, n, axes], or [n, axes] for all batches alike;
    packed tensors [total, heads, d] take [total, axes].  ``inverse`` turns
    back: applied to the outputs' gradients it gives the inputs'.  Returns
    (q, k) as new contiguous tensors, or with ``inplace`` the given ones, which
    must not share elements and, in grad mode, not require gradients."""
    return rope_with(q, k, positions, plan, plan.fixed, inverse, inplace)


def rope_with(q, k, positions, plan, fixed, inverse=False, inplace=False):
    """``rope`` with the plan's frequencies in ``fixed``, a tensor on q's device."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype not in _lib.DTYPES:
        raise TypeError("q must be a bf16, fp16 or fp32 CUDA tensor")
    if q.dim() == 3:
        out = rope_with(q[None], None if k is None else k[None], positions, plan, fixed, inverse,
                        inplace)
        return (q, k) if inplace else (out[0][0], None if k is None else out[1][0])
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k are [B, n, heads, d] or packed [total, heads, d]")
    B, n, H, d = q.shape
    if d != plan.head_dim:
        raise ValueError(f"heads of {d} dimensions, the plan is for {plan.head_dim}")
    if H < 1:
        raise ValueError("q needs at least one head")
    dev, dtype = q.device, q.dtype
    _tensor(fixed, "plan", dev, torch.int64, (plan.pairs,))
    axes = len(plan.sections)
    batched = positions.dim() == 3
    _tensor(positions, "positions", dev, torch.int32, (B, n, axes) if batched else (n, axes))
    if inplace and torch.is_grad_enabled() and \
            (q.requires_grad or (k is not None and k.requires_grad)):
        raise ValueError("in place, the rotation would be missing from the gradients: use Rotary")
    none = (0, 0, 0)
    q_in, q_out = _rope_strides(q, "q", dtype, B, n, d), q
    if not inplace:
        q_out = torch.empty((B, n, H, d), dtype=dtype, device=dev)
    q_st = q_out.stride()[:3]
    Hk, k_ptr, k_out_ptr, k_in, k_st, k_out = 0, 0, 0, none, none, None
    if k is not None:
        Hk = k.shape[2]
        k_in, k_out = _rope_strides(k, "k", dtype, B, n, d), k
        if k.device != dev:
            raise ValueError(f"k is on {k.device}, expected {dev}")
        if not inplace:
            k_out = torch.empty((B, n, Hk, d), dtype=dtype, device=dev)
        k_st = k_out.stride()[:3]
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    # bl_rope_args, field by field
    args = _ROPE_ARGS.pack(
        B, n, H, Hk, d, plan.pairs, axes, *plan.padded_sections, plan.layout == "interleaved",
        bool(inverse), _lib.DTYPES[dtype], q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr,
        *q_in, *k_in, *q_st, *k_st, positions.data_ptr(), n * axes if batched else 0,
        fixed.data_ptr())
    _launch("bl_rope", dev, args)
    if inplace:                            # what autograd holds of them is stale now
        torch.autograd.graph.increment_version(q if k is None else (q, k))
    return q_out, k_out


_ROPE_ARGS = struct.Struct("<14i4Q12qQqQ")


def grid_positions(T, Y, X, device="cuda", dtype=torch.int32):
    """int32 [T * Y * X, 3] positions (t, y, x) of a grid flattened t-major."""
    i = torch.arange(T * Y * X, device=device)
    return torch.stack((i // (Y * X), i // X % Y, i % X), -1).to(dtype)
