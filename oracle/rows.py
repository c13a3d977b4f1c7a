"""Plain CPU forms of the row operators: the root-mean-square norm with the
residual's addition, rows in 8 bits, and the linear layer on packed int4
weights.  The ``*64`` functions evaluate the operators' formulas in binary64;
``codes32`` follows the documented binary32 order operation by operation, whose
codes are bit-exact.  No arithmetic is shared with the GPU side."""
from __future__ import annotations

import math

import numpy as np


def add64(x, residual=None):
    h = np.asarray(x, np.float64)
    return h if residual is None else h + np.asarray(residual, np.float64)


def rstd64(h, eps):
    return 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)


def norm64(x, weight, residual=None, eps=1e-6):
    h = add64(x, residual)
    return h * rstd64(h, eps) * np.asarray(weight, np.float64)


def scaled64(x, weight=None, residual=None, channel_scales=None):
    """t = h * weight * channel_scale, the values that 8 bits stand for up to
    the row's factor."""
    t = add64(x, residual)
    for f in (weight, channel_scales):
        if f is not None:
            t = t * np.asarray(f, np.float64)
    return t


def codes32(x, weight=None, residual=None, channel_scales=None):
    """Codes of rows given in binary32 (exact values of their type)."""
    t = np.asarray(x, np.float32)
    if residual is not None:
        t = t + np.asarray(residual, np.float32)
    for f in (weight, channel_scales):
        if f is not None:
            t = t * np.asarray(f, np.float32)
    peak = np.abs(t).max(axis=1, keepdims=True)
    dead = ~(peak >= np.float32(2.0 ** -100)) | ~np.isfinite(peak)
    with np.errstate(all="ignore"):
        codes = np.rint(t * (np.float32(127.0) / peak))
    return np.where(dead, 0, np.nan_to_num(codes)).astype(np.int8)


def unpack_int4(packed):
    """int4 values [N, K] of a packed matrix [N, K/2]."""
    p = np.asarray(packed).astype(np.int16)
    q = np.empty((p.shape[0], 2 * p.shape[1]), np.int64)
    for half, nibble in enumerate((p & 15, p >> 4)):
        q[:, half::2] = np.where(nibble >= 8, nibble - 16, nibble)
    return q


def activate64(y, activation):
    if activation == "relu":
        return np.where(y < 0, 0.0, y)
    if activation == "gelu":
        return 0.5 * y * np.vectorize(math.erfc, otypes=[np.float64])(-y * math.sqrt(0.5))
    if activation == "silu":
        with np.errstate(over="ignore"):
            return y / (1.0 + np.exp(-y))
    return y


def linear64(codes, row_scales, packed, out_scales=None, bias=None, activation=None, residual=None):
    """(result, value in front of the activation, products' scaled sums)."""
    # whole numbers far below 2^53: the binary64 products and sums are exact
    acc = np.asarray(codes, np.float64) @ unpack_int4(packed).T.astype(np.float64)
    s = acc * np.asarray(row_scales, np.float64)[:, None]
    if out_scales is not None:
        s = s * np.asarray(out_scales, np.float64)
    y = s if bias is None else s + np.asarray(bias, np.float64)
    z = activate64(y, activation)
    if residual is not None:
        z = z + np.asarray(residual, np.float64)
    return z, y, s
