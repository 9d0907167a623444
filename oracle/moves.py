"""Tokens to the experts' rows, and the gradients of that move and of the
weighted way back (combine.py).  TEST INFRASTRUCTURE ONLY (see the package
docstring).

    dispatch           A[row(t, j)] = x[t]
    dispatch_backward  dx[t] = bf16( sum_j dA[row(t, j)] ), fp32 in slot order from 0
    combine_backward   dC[row(t, j)] = bf16( fl32(w[t, j] * dout[t]) ),
                       dw[t, j] = sum_n C[row(t, j), n] dout[t, n]  (fp64 here)

Slots whose row is outside [0, R) move nothing and have dw = 0.  Every bf16
result is unique; dw is an fp32 sum on the device, compared under its bound.
"""

from __future__ import annotations

import numpy as np

from .combine import combine_ref
from .formats import bf16_bits_to_f64, bf16_rne_bits


def dispatch_ref(x_bits, row_of_slot, top_k: int, R: int, init=None) -> np.ndarray:
    x = np.asarray(x_bits, dtype=np.uint16)
    A = np.zeros((R, x.shape[1]), np.uint16) if init is None else np.array(init, dtype=np.uint16)
    for s, r in enumerate(np.asarray(row_of_slot, dtype=np.int64).reshape(-1)):
        if 0 <= r < R:
            A[r] = x[s // top_k]
    return A


def dispatch_backward_ref(dA_bits, row_of_slot, T: int, top_k: int) -> np.ndarray:
    return combine_ref(dA_bits, row_of_slot, np.ones(T * top_k, np.float32), T, top_k)


def combine_backward_ref(C_bits, dout_bits, row_of_slot, weights, T: int, top_k: int, init=None):
    """(dC bf16 bits [R, N], dw fp64 [T*top_k], the magnitude sums of dw's products)."""
    C = bf16_bits_to_f64(C_bits)
    d = bf16_bits_to_f64(dout_bits)
    R, N = C.shape
    w = np.asarray(weights, dtype=np.float32).reshape(-1)
    dC = np.zeros((R, N), np.uint16) if init is None else np.array(init, dtype=np.uint16)
    dw, mag = np.zeros(T * top_k), np.zeros(T * top_k)
    for s, r in enumerate(np.asarray(row_of_slot, dtype=np.int64).reshape(-1)):
        if 0 <= r < R:
            g = d[s // top_k]
            dC[r] = bf16_rne_bits((w[s] * g.astype(np.float32)).astype(np.float64))
            dw[s] = float((C[r] * g).sum())
            mag[s] = float(np.abs(C[r] * g).sum())
    return dC, dw, mag
