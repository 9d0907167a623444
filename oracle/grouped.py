"""The products grouped by expert and their gradients, and the scaling of
gradients by their norm, in fp64.  TEST INFRASTRUCTURE ONLY (see the package
docstring).

    C[r] = A[r] W[e]^T,  dA[r] = dC[r] W[e],  dW[e] = sum over the rows r of e of dC[r]^T A[r]
    norm = sqrt(sum x^2),  out = min(1, max_norm / (norm + eps)) x

Each product also comes with absolute=True: the sum of the products'
magnitudes, by which an fp32 sum's roundings are counted.  Rows outside every
expert are NaN here (nothing is written there).
"""

from __future__ import annotations

import math

import numpy as np


def _rows(offsets):
    off = np.asarray(offsets, dtype=np.int64)
    return [(e, slice(off[e], off[e + 1])) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def _v(x, absolute):
    return np.abs(x) if absolute else x


def forward_f64(A, W, offsets, absolute=False):
    out = np.full((A.shape[0], W.shape[1]), np.nan)
    for e, r in _rows(offsets):
        out[r] = _v(A[r], absolute) @ _v(W[e], absolute).T
    return out


def dgrad_f64(dC, W, offsets, absolute=False):
    out = np.full((dC.shape[0], W.shape[2]), np.nan)
    for e, r in _rows(offsets):
        out[r] = _v(dC[r], absolute) @ _v(W[e], absolute)
    return out


def wgrad_f64(dC, A, offsets, absolute=False):
    out = np.zeros((len(offsets) - 1, dC.shape[1], A.shape[1]))
    for e, r in _rows(offsets):
        out[e] = _v(dC[r], absolute).T @ _v(A[r], absolute)
    return out


def clip_f64(tensors, max_norm, eps):
    """(norm, coefficient, scaled tensors)."""
    norm = math.sqrt(math.fsum(float(np.sum(np.square(np.asarray(t, dtype=np.float64)))) for t in tensors))
    c = min(1.0, float(np.float32(max_norm)) / (norm + float(np.float32(eps))))
    return norm, c, [np.asarray(t, dtype=np.float64) * c for t in tensors]
