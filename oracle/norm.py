"""Root-mean-square norm with the residual's addition, its 8-bit output and its
gradient, in fp64.  TEST INFRASTRUCTURE ONLY (see the package docstring).

    h = bf16(x + r),  n = (mean(h^2) + eps)^(-1/2),  y = h n w
    dx = n (g - h n mean(g h n)) + dsum, g = dy w,   dw = sum over rows of dy h n

h is unique (the fp32 sum of two bf16 values rounded to bf16).  y, dx and dw
are the definitions; `check_codes` says whether 8-bit codes and scales are
those of a y within a relative distance of the definition's.
"""

from __future__ import annotations

import numpy as np

from .formats import bf16_bits_to_f64, bf16_rne_bits, e4m3_table


def sum_bits(x_bits, res_bits=None) -> np.ndarray:
    """h: the sum in fp32 (one rounding), then to bf16."""
    x = bf16_bits_to_f64(x_bits)
    if res_bits is None:
        return np.asarray(x_bits, dtype=np.uint16)
    with np.errstate(over="ignore", invalid="ignore"):
        s = (x.astype(np.float32) + bf16_bits_to_f64(res_bits).astype(np.float32)).astype(np.float64)
    return bf16_rne_bits(s)


def _inv(h, eps):
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        return 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + np.float64(np.float32(eps)))


def rms_norm_f64(h_bits, w, eps) -> np.ndarray:
    h = bf16_bits_to_f64(h_bits)
    with np.errstate(invalid="ignore", over="ignore"):
        return h * _inv(h, eps) * (1.0 if w is None else np.asarray(w, dtype=np.float64))


def rms_norm_backward_f64(h_bits, w, dy_bits, eps, dsum_bits=None):
    """(dx, dw, and per element the magnitudes n (|g| + |h n| mean|g h n|) + |dsum| and sum |dy h n| that
    roundings are counted by)."""
    h, dy = bf16_bits_to_f64(h_bits), bf16_bits_to_f64(dy_bits)
    n = _inv(h, eps)
    xh = h * n
    g = dy * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    dx = n * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    mag = n * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    if dsum_bits is not None:
        r = bf16_bits_to_f64(dsum_bits)
        dx, mag = dx + r, mag + np.abs(r)
    return dx, np.sum(dy * xh, axis=0), mag, np.sum(np.abs(dy * xh), axis=0)


def e4m3_nearest(v) -> np.ndarray:
    """Values of the E4M3FN grid nearest to v (|v| <= 448 (1 + 2^-20)), halves to the even code."""
    grid = np.unique(np.abs(e4m3_table()[:127]))            # ascending, index = code
    a = np.minimum(np.abs(np.asarray(v, dtype=np.float64)), 448.0)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))   # on a midpoint: the even one
    return np.copysign(grid[code], v)


def check_codes(codes, scales, y, rel) -> int:
    """Wrong codes or scales: codes uint8 [T, K], scales fp32 [T, K/128] of y fp64 [T, K], where the device's y may
    be off by `rel` (and its amax / 448, its reciprocal and the product by another 2^-22)."""
    T, K = y.shape
    yg = y.reshape(T, K // 128, 128)
    s = np.asarray(scales, dtype=np.float64)
    a = np.abs(yg).max(axis=2)
    want = np.where(a < 2.0 ** -100, 1.0, a / 448.0)
    wrong = int(np.count_nonzero(~(np.abs(s - want) <= want * (rel + 2.0 ** -22))))
    v = e4m3_table()[np.asarray(codes)].reshape(yg.shape)
    q, slack = yg / s[:, :, None], rel + 2.0 ** -22
    lo, hi = e4m3_nearest(q * (1 - np.sign(q) * slack)), e4m3_nearest(q * (1 + np.sign(q) * slack))
    return wrong + int(np.count_nonzero(~((v >= np.minimum(lo, hi)) & (v <= np.maximum(lo, hi)))))
