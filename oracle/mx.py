"""Numpy oracle of the operators on MXFP4 tensors — test infrastructure only.

Plain float64 transcriptions of the definitions in include/svdq.h (svdq_mx_*): the block rule and the
codes are those of `quantize_mx` (the msModelSlim SVDQuant guide, step 2: MXFP4 per block, min-max);
a gated feed-forward block multiplies act(g) by u.
"""
from __future__ import annotations

import math

import numpy as np

from .svdquant import MX_BLOCK, dequant_mx, quantize_mx

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def quantize(x):
    """(codes [rows, K], scale bytes [rows, blocks]): quantize_mx, and byte 255 with zero codes for a block
    that holds an infinity or a NaN."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    nb = -(-K // MX_BLOCK)
    padded = np.zeros((rows, nb * MX_BLOCK))
    padded[:, :K] = x
    bad = ~np.isfinite(padded.reshape(rows, nb, MX_BLOCK)).all(-1)
    mask = np.repeat(bad, MX_BLOCK, axis=1)[:, :K]
    codes, sbytes = quantize_mx(np.where(mask, 0.0, x))
    return np.where(mask, 0, codes).astype(np.uint8), np.where(bad, 255, sbytes).astype(np.uint8)


def dequantize(codes, sbytes):
    nan = np.repeat(np.asarray(sbytes) == 255, MX_BLOCK, axis=1)[:, : np.asarray(codes).shape[1]]
    return np.where(nan, np.nan, dequant_mx(codes, np.where(np.asarray(sbytes) == 255, 127, sbytes)))


def values(x):
    """Q(x): the values that stand for x, quantised along its rows."""
    return dequantize(*quantize(x))


def unpack(codes_bytes, scale_bytes, rows, K):
    """(codes [rows, K], scale bytes [rows, blocks], codes past K, scale bytes past K) of the library's tiled
    arrays: codes in 16-row x 128-code tiles of 1 KB, scales in 64-row x 4-block tiles of 256 bytes."""
    kq = 2 * -(-K // 256)
    r16, r64 = -(-rows // 16), -(-rows // 64)
    b = np.asarray(codes_bytes).reshape(r16, kq, 16, 64).transpose(0, 2, 1, 3).reshape(r16 * 16, kq * 64)[:rows]
    codes = np.stack([b & 15, b >> 4], axis=-1).reshape(rows, kq * 128)
    s = np.asarray(scale_bytes).reshape(r64, kq, 64, 4).transpose(0, 2, 1, 3).reshape(r64 * 64, kq * 4)[:rows]
    nb = -(-K // MX_BLOCK)
    return codes[:, :K], s[:, :nb], codes[:, K:], s[:, nb:]


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(name, g):
    """act(g)."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        if name == "silu":
            return g / (1 + np.exp(-g))
        if name == "gelu":
            return g * 0.5 * _erfc(-g / math.sqrt(2))
        if name == "gelu_tanh":
            # (1 + tanh z) / 2 = 1 / (1 + e^(-2 z)), which keeps its digits for negative z
            return g / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g**3)))
    return np.maximum(g, 0.0)


def act_grad(name, g):
    """act'(g)."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        if name == "silu":
            s = 1 / (1 + np.exp(-g))
            return s * (1 + g * (1 - s))
        if name == "gelu":
            return 0.5 * _erfc(-g / math.sqrt(2)) + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":
            c = math.sqrt(2 / math.pi)
            s = 1 / (1 + np.exp(-2 * c * (g + 0.044715 * g**3)))
            return s * (1 + g * (1 - s) * 2 * c * (1 + 3 * 0.044715 * g * g))
    return (g > 0).astype(np.float64)


def gated_grad(dh, gu, name):
    """[dg | du] of h = act(g) * u, gu = [g | u]."""
    dh, gu = np.asarray(dh, np.float64), np.asarray(gu, np.float64)
    F = dh.shape[1]
    g, u = gu[:, :F], gu[:, F:]
    return np.concatenate([dh * u * act_grad(name, g), dh * act(name, g)], axis=1)
