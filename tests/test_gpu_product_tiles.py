"""The kernels of every tile of the grouped products on the GPU, over the cases of
product_cases.py (whose tiles test_product_tiles.py asserts), random values,
against oracle/grouped.py.

Bounds.  bf16: products are exact in fp32 and a sum of Z of them in any order is
within (Z + 8) 2^-23 of the magnitudes' sum, then one rounding to bf16 (2^-8) or
fp32 (2^-24).  4 by 4 bits: helpers.fp32_sum_eps (the matrix core's sum of 128
products, one fp32 rounding per 128)."""

import numpy as np
import pytest
import torch

from helpers import GROUP_EPS_RANDOM_CODES, fp32_sum_eps
from oracle import bf16_bits_to_f64, bf16_rne_bits, fp4, grouped
from product_cases import CASES, FORWARD, FOUR_BITS, ROW_GRADIENT

pytestmark = pytest.mark.gpu


def _draw(rng, *shape):
    b = bf16_rne_bits(rng.standard_normal(shape, dtype=np.float32).astype(np.float64))
    return b, bf16_bits_to_f64(b)


def _dev(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def _near(got, want, err, half):
    g = got.double().cpu().numpy()
    bound = err + half * (np.abs(want) + err) + 2.0 ** -134
    assert np.all(np.isfinite(g))
    worst = float(np.max(np.abs(g - want) / bound))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("product,counts,N,K", [c[:4] for c in CASES if c[0] != FOUR_BITS])
def test_bf16(gpu_lib, product, counts, N, K):
    rng = np.random.default_rng(N + K)
    R, E, extra = sum(counts), len(counts), 3
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    off = torch.from_numpy(offs).cuda()
    if product in (FORWARD, ROW_GRADIENT):
        A, Af = _draw(rng, R + extra, K if product == FORWARD else N)
        W, Wf = _draw(rng, E, N, K)
        A[R:] = 0x7FC0                                  # rows behind the last expert are not touched
        call, ref = ((gpu_lib.grouped_gemm_bf16, grouped.forward_f64) if product == FORWARD else
                     (gpu_lib.grouped_gemm_dgrad, grouped.dgrad_f64))
        out = torch.full((R + extra, N if product == FORWARD else K), 7.0, dtype=torch.bfloat16, device="cuda")
        call(_dev(A), _dev(W), off, out=out)
        assert (out[R:] == 7.0).all()
        Z = A.shape[1]
        _near(out[:R], ref(Af[:R], Wf, offs), (Z + 8) * 2.0 ** -23 * ref(Af[:R], Wf, offs, absolute=True), 2.0 ** -8)
        return
    (dC, dCf), (A, Af) = _draw(rng, R, N), _draw(rng, R, K)
    want = grouped.wgrad_f64(dCf, Af, offs)
    err = (max(counts) + 8) * 2.0 ** -23 * grouped.wgrad_f64(dCf, Af, offs, absolute=True)
    _near(gpu_lib.grouped_gemm_wgrad(_dev(dC), _dev(A), off), want, err, 2.0 ** -24)
    out = torch.full((E, N, K), 5.0, dtype=torch.bfloat16, device="cuda")
    _near(gpu_lib.grouped_gemm_wgrad(_dev(dC), _dev(A), off, out=out), want, err, 2.0 ** -8)


@pytest.mark.parametrize("counts,N,K", [c[1:4] for c in CASES if c[0] == FOUR_BITS])
def test_four_bits(gpu_lib, counts, N, K):
    rng = np.random.default_rng(N + K)
    R, E = sum(counts), len(counts)
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    off = torch.from_numpy(offs).cuda()
    c = lambda v: torch.from_numpy(v).cuda()
    A = rng.integers(0, 256, (R, K // 2), dtype=np.uint8)
    B = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    # scales over 4 and 12 binades each: neighbours along z, rows and columns differ
    for lo, hi, eps in ((126, 130, 2.0 ** -16), (120, 132, GROUP_EPS_RANDOM_CODES)):
        SA = rng.integers(lo, hi, (R, K // 32), dtype=np.uint8)
        SB = rng.integers(lo, hi, (E, N, K // 32), dtype=np.uint8)
        out = torch.full((R + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
        pad = lambda v: np.concatenate([v, np.full((3, v.shape[1]), 255, np.uint8)])
        gpu_lib.grouped_gemm_a4(c(pad(A)), c(pad(SA)), c(B), c(SB), off, out=out)
        assert (out[R:] == 7.0).all()
        Af, Bf = fp4.decode_f64(A, SA, False), fp4.decode_f64(B, SB, False)
        _near(out[:R], grouped.forward_f64(Af, Bf, offs),
              fp32_sum_eps(K, eps) * grouped.forward_f64(Af, Bf, offs, absolute=True), 2.0 ** -8)
