"""Products of a few tokens with 4-bit weights and group scales, in fp64.
TEST INFRASTRUCTURE ONLY (see the package docstring).

    y[s, n] = gs[e] sum_k x[s // (S / X), k] (q(e, n, k) - z(e, n, k // group)) sc(e, n, k // group)

e = ids[s] (0 without ids); a slot whose id is outside [0, E) is all zeros.
MXFP4 and NVFP4 weights decode as in a16.py (q an E2M1 value, no zero point);
INT4: q the code 0 .. 15, z the zero point (8 if none are given), sc bf16.
"""

from __future__ import annotations

import numpy as np

from .a16 import FMT_MX, FMT_NV, _np, decode_weights_a16
from .formats import bf16_bits_to_f64

FMT_INT4 = 2


def decode_int4(b_packed, scale_bits, zeros) -> np.ndarray:
    """codes uint8 [N, K/2], bf16 bits [N, K/group], zeros uint8 [N, K/group] or None -> fp64 [N, K]."""
    b = _np(b_packed).astype(np.int64)
    q = np.stack([b & 15, b >> 4], axis=2).reshape(b.shape[0], -1).astype(np.float64)
    sc = bf16_bits_to_f64(_np(scale_bits).view(np.uint16))
    z = np.full(sc.shape, 8.0) if zeros is None else _np(zeros).astype(np.float64)
    group = q.shape[1] // sc.shape[1]
    return (q - np.repeat(z, group, axis=1)) * np.repeat(sc, group, axis=1)


def matvec_f64(x_bits, B, SB, fmt: int, ids=None, gs=None, zeros=None, S: int | None = None):
    """(y fp64 [S, N], the sums of the products' magnitudes)."""
    x = bf16_bits_to_f64(x_bits)
    B, SB = _np(B), _np(SB)
    E, N = B.shape[0], B.shape[1]
    X = x.shape[0]
    experts = np.zeros(X, np.int64) if ids is None else _np(ids).astype(np.int64).reshape(-1)
    S = len(experts)
    y, mag = np.zeros((S, N)), np.zeros((S, N))
    cache = {}
    for s, e in enumerate(experts):
        if not 0 <= e < E:
            continue
        if e not in cache:
            cache[e] = (decode_int4(B[e], SB[e], None if zeros is None else _np(zeros)[e]) if fmt == FMT_INT4
                        else decode_weights_a16(B[e], SB[e], fmt))
        W, xs = cache[e], x[s // (S // X)]
        g = 1.0 if gs is None else float(np.float32(_np(gs)[e]))
        y[s] = (W @ xs) * g
        mag[s] = (np.abs(W) @ np.abs(xs)) * abs(g)
    return y, mag


__all__ = ["FMT_INT4", "FMT_MX", "FMT_NV", "decode_int4", "matvec_f64"]
