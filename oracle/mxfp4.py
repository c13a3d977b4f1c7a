"""Plain CPU forms of rows in microscaled 4-bit floating point (32 channels
share a power of two) and of the linear layer between two such matrices.
numpy, no arithmetic shared with the GPU side."""
from __future__ import annotations

import numpy as np

from oracle import rows

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes uint8 [M, H/2], scales uint8 [M, H/32]) of rows given exactly."""
    x = np.asarray(x, np.float64)
    v = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[..., None], 0.0, v)
    peak = np.abs(v).max(axis=2)
    # frexp: peak = f * 2^e with f in [0.5, 1)
    s = np.clip(np.frexp(peak)[1] - 1 - 2 + 127, 0, 254)
    s = np.where(peak > 0, s, 0)
    t = np.ldexp(np.abs(v), (127 - s)[..., None])        # exact
    # the nearest value; of two as near, the even code
    d = np.abs(t[..., None] - VALUES)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    code = code + 8 * np.signbit(v)
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, s).astype(np.uint8)


def values(codes, scales):
    """The values in 64 bits, NaN under a scale of 255."""
    codes = np.asarray(codes)
    q = np.empty((codes.shape[0], 2 * codes.shape[1]), np.int64)
    q[:, 0::2], q[:, 1::2] = codes & 15, codes >> 4
    v = VALUES[q & 7] * np.where(q >= 8, -1.0, 1.0)
    s = np.asarray(scales, np.int64)
    v = np.ldexp(v.reshape(codes.shape[0], -1, 32), (s - 127)[..., None])
    return np.where((s == 255)[..., None], np.nan, v).reshape(codes.shape[0], -1)


def linear64(codes, scales, w_codes, w_scales, bias=None, activation=None, residual=None):
    """(result, value in front of the activation, the products' sum of
    magnitudes)."""
    x, w = values(codes, scales), values(w_codes, w_scales)
    y = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    z = rows.activate64(y, activation)
    if residual is not None:
        z = z + np.asarray(residual, np.float64)
    return z, y, size
