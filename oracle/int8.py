"""Numpy oracle of the operators on 8-bit tensors with row scales and of layer norm — test infrastructure only.

Plain float64 transcriptions of the definitions in include/svdq.h (svdq_i8_*, svdq_layer_norm*).
"""
from __future__ import annotations

import numpy as np


def quantize(x):
    """(codes [rows, K], scales [rows] in float32) of each row. The quotients are float64's: a quotient of two float32 values that
    is no tie differs from one by far more than float64 rounds."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(1)
    z = np.where(bad[:, None], 0.0, x)
    most = np.abs(z).max(1)
    s = np.where(most > 0, np.maximum((most / 127).astype(np.float32), np.float32(2.0**-126)), 0).astype(np.float32)
    codes = np.rint(z / np.where(s == 0, 1, s).astype(np.float64)[:, None])
    return codes.astype(np.int8), np.where(bad, np.nan, s).astype(np.float32)


def dequantize(codes, scales):
    return np.asarray(codes, np.float64) * np.asarray(scales, np.float64)[:, None]


def values(x):
    """Q(x): the values that stand for x, quantised along its rows."""
    return dequantize(*quantize(x))


def unpack(code_bytes, rows, K):
    """(codes [rows, K], codes past K) of the library's tiles of 16 rows x 64 codes."""
    kq, r16 = 2 * -(-K // 128), -(-rows // 16)
    c = np.asarray(code_bytes).view(np.int8).reshape(r16, kq, 16, 64).transpose(0, 2, 1, 3).reshape(r16 * 16, kq * 64)[:rows]
    return c[:, :K], c[:, K:]


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    y = y if weight is None else y * np.asarray(weight, np.float64)
    return (y if bias is None else y + np.asarray(bias, np.float64)), mean, rstd


def layer_norm_grad(dy, x, mean, rstd, weight=None):
    """(dx, dweight, dbias)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
