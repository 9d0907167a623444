"""SwiGLU with an 8-bit copy of its input, and its gradient from that copy.
TEST INFRASTRUCTURE ONLY (see the package docstring).

    copy: per (row, 128 columns of C): a = max|C| (NaN left out),
          s = fl32(a / 448), 1 where a < 2^-100, code = E4M3FN RNE of
          fl32(C * fl32(1 / s)); a NaN element keeps a NaN code.
    dg = dh u s (1 + g (1 - s)),  du = dh g s,  h = g s u,  s = 1 / (1 + e^-g),
    with g, u = code * scale.

The copy's bits are unique; the gradients are the definition in fp64.
"""

from __future__ import annotations

import numpy as np

from .formats import e4m3_table
from .quant import bf16_bits_to_f32, e4m3_encode_rne

_LUT8 = e4m3_table()


def checkpoint_ref(C_bits):
    """bf16 bits [R, W] (finite) -> (codes uint8 [R, W], scales fp32 [R, W/128])."""
    x = bf16_bits_to_f32(C_bits)
    R, W = x.shape
    xg = x.reshape(R, W // 128, 128)
    a = np.max(np.abs(xg), axis=2)
    s = np.where(a < np.float32(2.0 ** -100), np.float32(1.0), a / np.float32(448.0)).astype(np.float32)
    inv = (np.float32(1.0) / s).astype(np.float32)
    y = (xg * inv[:, :, None]).astype(np.float32)
    # values a rounding above 448 belong to code 448
    return e4m3_encode_rne(np.clip(y, np.float32(-448.0), np.float32(448.0))).reshape(R, W), s


def decode_f64(codes, scales) -> np.ndarray:
    codes = np.asarray(codes, dtype=np.uint8)
    return _LUT8[codes] * np.repeat(np.asarray(scales, dtype=np.float64).reshape(codes.shape[0], -1), 128, axis=1)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu_backward_f64(codes, scales, dh):
    """(dC fp64 [R, 2I], h fp64 [R, I])."""
    v = decode_f64(codes, scales)
    I = v.shape[1] // 2
    g, u = v[:, :I], v[:, I:]
    dh = np.asarray(dh, dtype=np.float64)
    s = _sigmoid(g)
    return np.concatenate([dh * u * s * (1.0 + g * _sigmoid(-g)), dh * g * s], axis=1), g * s * u
