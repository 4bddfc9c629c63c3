"""Plain CPU oracle for the operators around the attention: rotary positions
with several axes, the root-mean-square norm with the residual's addition, and
activations in 8 bits.

TEST INFRASTRUCTURE ONLY (see the package).  fp64 numpy, written from the
definitions; the 8-bit codes are defined by a few fp32 roundings, which numpy
float32 performs one by one, so they can be compared bit for bit.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


# --- rotary positions ------------------------------------------------------------

def rope(x, positions, sections, freqs, interleaved, inverse=False):
    """x [B, n, heads, d]; positions [B, n, axes]; pair p of section a turns by
    positions[..., a] * freqs[p]."""
    x = _f64(x).copy()
    positions = np.asarray(positions, dtype=np.int64)
    pairs = sum(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    for p in range(pairs):
        angle = positions[..., axis[p]].astype(np.longdouble) * np.longdouble(freqs[p])
        if inverse:
            angle = -angle
        c = np.cos(angle).astype(np.float64)[..., None]
        s = np.sin(angle).astype(np.float64)[..., None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
        u, v = x[..., i].copy(), x[..., j].copy()
        x[..., i] = u * c - v * s
        x[..., j] = u * s + v * c
    return x


# --- root-mean-square norm -------------------------------------------------------

def rms_norm(x, weight, eps, residual=None):
    """(y, h, rstd) of [rows, cols]."""
    h = _f64(x) if residual is None else _f64(x) + _f64(residual)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    w = 1.0 if weight is None else _f64(weight)
    return h * rstd[:, None] * w, h, rstd


def rms_norm_backward(g_y, h, rstd, weight, g_h=None):
    """(g_x, g_w) of [rows, cols] from the given h and rstd."""
    g_y, h, rstd = _f64(g_y), _f64(h), _f64(rstd)
    w = np.ones(h.shape[1]) if weight is None else _f64(weight)
    u = h * rstd[:, None]
    c = (w * g_y * u).mean(axis=1, keepdims=True)
    g_x = rstd[:, None] * (w * g_y - u * c)
    if g_h is not None:
        g_x = g_x + _f64(g_h)
    return g_x, (g_y * u).sum(axis=0)


# --- activations in 8 bits -------------------------------------------------------

def e4m3_values():
    """The value of every e4m3 code 0 .. 255 (the two NaN codes as NaN): sign, 4
    exponent bits with bias 7, 3 mantissa bits; no infinities."""
    out = []
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        e, m = (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            out.append(np.nan)
        elif e == 0:
            out.append(sign * m * 2.0 ** -9)
        else:
            out.append(sign * (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


def round_e4m3(x):
    """Codes (uint8) of the nearest values, ties to the even code."""
    values = e4m3_values()[:127]                  # 0 .. 448, ascending with the code
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.minimum(np.searchsorted(values, a), 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - values[lo], values[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def save8(x, fmt, group):
    """(codes, scales) of [rows, cols] values that fp32 holds; codes int8 or
    uint8 bits of e4m3."""
    x = np.asarray(_f64(x), dtype=np.float32)
    rows, cols = x.shape
    size = group or cols
    groups = -(-cols // size)
    qmax = np.float32(127.0 if fmt == "int8" else 448.0)
    codes = np.zeros((rows, cols), dtype=np.int8 if fmt == "int8" else np.uint8)
    scales = np.zeros((rows, groups), dtype=np.float32)
    for g in range(groups):
        part = x[:, g * size:(g + 1) * size]
        bad = ~np.isfinite(part).all(axis=1)
        amax = np.abs(np.where(bad[:, None], 0, part)).max(axis=1)
        scale = np.maximum(amax * (np.float32(1) / qmax), np.float32(2.0 ** -126))
        top = np.float32(float(np.finfo(np.float32).max) / float(qmax))
        if float(top) * float(qmax) > float(np.finfo(np.float32).max):
            top = np.nextafter(top, np.float32(0))
        scale = np.minimum(scale, top)
        q = np.where(bad[:, None], np.float32(0), part) * (np.float32(1) / scale)[:, None]
        assert q.dtype == np.float32
        codes[:, g * size:(g + 1) * size] = np.rint(q) if fmt == "int8" else round_e4m3(q)
        codes[bad, g * size:(g + 1) * size] = 0
        scales[:, g] = np.where(bad, np.float32(np.nan), scale)
    return codes, scales


def load8(codes, scales, group):
    """fp64 values of codes (int8, or uint8 bits of e4m3)."""
    v = e4m3_values()[codes] if codes.dtype == np.uint8 else codes.astype(np.float64)
    cols = codes.shape[1]
    return v * np.repeat(scales.astype(np.float64), group or cols, axis=1)[:, :cols]
