"""Plain CPU oracle for the linear layers around the attention: products of 8-bit
codes with block scales, the layer norm, and dropout from a counter-based
generator.

TEST INFRASTRUCTURE ONLY (see the package).  fp64 numpy, written from the
definitions; codes are defined by a few fp32 roundings, and the generator by
whole numbers, so both can be compared bit for bit.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64


# --- layer norm ------------------------------------------------------------------

def layer_norm(x, weight, bias, eps, residual=None):
    """(y, h, mean, rstd) of [rows, cols]."""
    h = _f64(x) if residual is None else _f64(x) + _f64(residual)
    mean = h.mean(axis=1)
    c = h - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * rstd[:, None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, h, mean, rstd


def layer_norm_backward(g_y, h, mean, rstd, weight, g_h=None):
    """(g_x, g_w, g_b) of [rows, cols] from the given h, mean and rstd."""
    g_y, rstd = _f64(g_y), _f64(rstd)[:, None]
    u = (_f64(h) - _f64(mean)[:, None]) * rstd
    wg = g_y if weight is None else g_y * _f64(weight)
    g_x = rstd * (wg - wg.mean(axis=1, keepdims=True) - u * (wg * u).mean(axis=1, keepdims=True))
    if g_h is not None:
        g_x = g_x + _f64(g_h)
    return g_x, (g_y * u).sum(axis=0), g_y.sum(axis=0)


# --- 8 bits ----------------------------------------------------------------------

def e4m3_values(codes):
    """Values of e4m3 bytes: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(c & 128, -v, v)


def block_scales(x, down, along):
    """fp32 scales of x [rows, cols] for every down x along elements (ends may be cut)."""
    x = np.abs(np.asarray(x, dtype=np.float32))
    rows, cols = x.shape
    out = np.empty((-(-rows // down), -(-cols // along)), dtype=np.float32)
    inv = np.float32(1) / np.float32(448)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            top = x[i * down:(i + 1) * down, j * along:(j + 1) * along].max()
            out[i, j] = max(np.float32(top * inv), np.float32(2.0 ** -126))
    return out


def spread(scales, down, along, rows, cols):
    """The scale of every element."""
    return np.repeat(np.repeat(scales, down, 0)[:rows], along, 1)[:, :cols]


def encode(x, scale):
    """e4m3 values (not bytes) of fp32 x under fp32 scales of its elements: the nearest of
    fl(x * fl(1 / scale)), ties to even."""
    inv = np.float32(1) / np.asarray(scale, dtype=np.float32)
    r = (np.asarray(x, dtype=np.float32) * inv).astype(np.float64)
    _, e = np.frexp(r)
    step = np.ldexp(1.0, np.maximum(e, -5) - 4)
    return np.clip(np.rint(r / step) * step, -448, 448)


# --- dropout ---------------------------------------------------------------------

def philox(counter, key):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011) of one counter of four 32-bit
    words and a key of two, in Python's whole numbers."""
    c, k = [int(x) for x in counter], [int(x) for x in key]
    low = 0xFFFFFFFF
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & low, (p >> 32) ^ c[3] ^ k[1], p & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def kept(n, p, seed, offset, first=0):
    """Whether elements first .. first + n - 1 are kept."""
    low = 0xFFFFFFFF
    out = np.empty(n, dtype=bool)
    words, at = None, None
    for i in range(n):
        j = (first + i) // 4
        if j != at:
            words = philox((j & low, j >> 32, offset & low, (offset >> 32) & low),
                           (seed & low, (seed >> 32) & low))
            at = j
        out[i] = words[(first + i) % 4] >= round(p * 2 ** 32)
    return out
