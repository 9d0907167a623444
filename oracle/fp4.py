"""bf16 to MXFP4 and NVFP4 and back.  TEST INFRASTRUCTURE ONLY (see the package
docstring).

    MX  e = floor(log2 amax) - 2 (>= -127), scale code e + 127 (127 for a group of zeros)
    NV  gs = fp32(amax of the expert / 2688), 1 below 2^-100; s = E4M3 of amax / (6 gs)
    code = E2M1 of x / scale: nearest, halves to the even code, past 6 to 6
A group with an infinity or a NaN: NaN scale, codes 0, outside the expert's amax.

Every decision is a comparison of x with a midpoint times the scale, whose
product is exact in fp64 (3 + 4 + 24 bits), so the result is unique.
"""

from __future__ import annotations

import numpy as np

from .formats import E2M1_VALUES, bf16_bits_to_f64, e2m1_table, e4m3_table, e8m0_value


def _nearest_code(a, grid, scale):
    """Index of the grid value nearest to a / scale (a, scale > 0), halves to the even index."""
    code = np.zeros(a.shape, dtype=np.int64)
    for i in range(len(grid) - 1):
        m = (grid[i] + grid[i + 1]) / 2 * scale
        code += (a > m) | ((a == m) & (i % 2 == 1))
    return code


def _codes(xg, scale):
    """E2M1 codes of xg / scale, sign bit kept; scale 0 gives zeros."""
    s = np.broadcast_to(scale, xg.shape)
    mag = np.where(s > 0, _nearest_code(np.abs(xg), np.array(E2M1_VALUES), np.where(s > 0, s, 1.0)), 0)
    return (mag | (np.signbit(xg).astype(np.int64) << 3)).astype(np.uint8)


def pack(codes) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed) -> np.ndarray:
    q = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), np.uint8)
    q[..., 0::2], q[..., 1::2] = packed & 15, packed >> 4
    return q


def quantize_mx(bits):
    """uint16 bf16 bits [.., K] -> (packed [.., K/2], E8M0 codes [.., K/32])."""
    x = bf16_bits_to_f64(bits)
    xg = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(xg).all(axis=-1)
    a = np.abs(np.where(bad[..., None], 0.0, xg)).max(axis=-1)
    e = np.where(a > 0, np.maximum(np.frexp(a)[1] - 3, -127), 0)
    codes = _codes(np.where(bad[..., None], 0.0, xg), np.ldexp(1.0, e)[..., None])
    codes[bad] = 0
    return pack(codes.reshape(x.shape)), np.where(bad, 255, e + 127).astype(np.uint8)


def quantize_nv(bits):
    """uint16 bf16 bits [E, N, K] -> (packed, E4M3 codes [E, N, K/16], fp32 [E])."""
    x = bf16_bits_to_f64(bits)
    xg = x.reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(xg).all(axis=-1)
    top = np.abs(np.where(np.isfinite(x), x, 0.0)).reshape(x.shape[0], -1).max(axis=1)
    gs = np.where(top < 2.0 ** -100, np.float32(1), top.astype(np.float32) / np.float32(2688)).astype(np.float32)
    g = gs.astype(np.float64)[:, None, None]
    xg = np.where(bad[..., None], 0.0, xg)
    a = np.abs(xg).max(axis=-1)
    grid = e4m3_table()[:127]
    sc = _nearest_code(a, grid, np.broadcast_to(6.0 * g, a.shape))
    codes = _codes(xg, (grid[sc] * g)[..., None])
    codes[bad] = 0
    return pack(codes.reshape(x.shape)), np.where(bad, 0x7F, sc).astype(np.uint8), gs


def decode_f64(packed, scales, nv: bool, gs=None) -> np.ndarray:
    """Values in fp64: [.., K]; gs fp32 [E] over the first dimension."""
    v = e2m1_table()[unpack(np.asarray(packed))]
    s = e4m3_table()[np.asarray(scales)] if nv else e8m0_value(scales)
    v = v * np.repeat(s, 16 if nv else 32, axis=-1)
    return v if gs is None else v * np.asarray(gs, dtype=np.float64).reshape(-1, *([1] * (v.ndim - 1)))


def gather_mx(x_bits, row_of_slot, top_k: int, R: int, A0, SA0):
    """Tokens in MXFP4 at the rows of their slots; A0, SA0: what rows without one hold."""
    q, s = quantize_mx(x_bits)
    A, SA = np.array(A0), np.array(SA0)
    for i, r in enumerate(np.asarray(row_of_slot).reshape(-1)):
        if 0 <= r < R:
            A[r], SA[r] = q[i // top_k], s[i // top_k]
    return A, SA
