"""The 4-bit quantiser, its inverse, the gather into grouped rows and the product
of 4-bit rows and weights on the GPU against oracle/fp4.py: codes and scales bit
for bit, values to one rounding (NVFP4: one in fp32 before it, 2^-24), products
within the bound of the grouped GEMM (helpers.fp32_sum_eps: the matrix core's
sum of 128 products, then one fp32 rounding per 128)."""

import numpy as np
import pytest
import torch

from helpers import GROUP_EPS_RANDOM_CODES, fp32_sum_eps
from oracle import bf16_bits_to_f64, bf16_rne_bits, fp4, grouped, route_ref

pytestmark = pytest.mark.gpu
MX, NV = 0, 1


def _dev(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _weights(E, N, K, seed):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((E, N, K)) * 0.02 * 2.0 ** rng.integers(-6, 7, (E, N, 1))
    v[rng.random((E, N, K)) < 0.02] = 0.0
    if N > 1:
        v[0, 1] = 0.0                                   # a row of zeros
    return bf16_rne_bits(v)


SHAPES = [(1, 1, 32), (1, 3, 64), (2, 5, 96), (3, 17, 128), (1, 300, 2048), (12, 33, 3584), (40, 2, 32), (2050, 1, 32)]


@pytest.mark.parametrize("E,N,K", SHAPES)
def test_quantize_and_back(gpu_lib, E, N, K):
    w = _weights(E, N, K, E + N + K)
    B, SB, none = gpu_lib.quantize_fp4(_dev(w), MX)
    q, s = fp4.quantize_mx(w)
    assert none is None and np.array_equal(SB.cpu().numpy(), s) and np.array_equal(B.cpu().numpy(), q)
    back = gpu_lib.dequantize_fp4(B, SB, MX)
    assert np.array_equal(_bits(back), bf16_rne_bits(fp4.decode_f64(q, s, False)))
    B, SB, gs = gpu_lib.quantize_fp4(_dev(w), NV)
    q, s, g = fp4.quantize_nv(w)
    assert np.array_equal(gs.cpu().numpy(), g) and np.array_equal(SB.cpu().numpy(), s)
    assert np.array_equal(B.cpu().numpy(), q)
    back = bf16_bits_to_f64(_bits(gpu_lib.dequantize_fp4(B, SB, NV, gs)))
    want = fp4.decode_f64(q, s, True, g)
    assert np.all(np.abs(back - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23))
    assert np.array_equal(_bits(gpu_lib.dequantize_fp4(B, SB, NV)), bf16_rne_bits(fp4.decode_f64(q, s, True)))


def test_every_mantissa_against_every_amax(gpu_lib):
    """All pairs of significands: x / scale meets every midpoint of both grids that bf16 weights can meet."""
    m = 1.0 + np.arange(128) / 128.0
    rows = []
    for a in m:                                          # amax a, the others at 5 binades below
        v = np.concatenate([m * s for s in (1.0, 0.5, 0.25, 0.125, 0.0625)])
        v = v[v <= a]
        v = np.pad(v, (0, -len(v) % 15))
        blocks = np.concatenate([np.full((len(v) // 15, 1), a), v.reshape(-1, 15)], axis=1).reshape(-1)
        rows.append(np.pad(blocks, (0, 768 - len(blocks))))
    v = np.stack(rows)                                   # one row per amax
    w = bf16_rne_bits(np.stack([v, -v])[:, :, None, :].reshape(2 * 128, 1, 768))   # an expert per amax
    B, SB, gs = gpu_lib.quantize_fp4(_dev(w), NV)
    q, s, g = fp4.quantize_nv(w)
    assert np.array_equal(gs.cpu().numpy(), g) and np.array_equal(SB.cpu().numpy(), s)
    assert np.array_equal(B.cpu().numpy(), q)
    w1 = w.reshape(1, 256, 768)                          # one expert: group scales spread under its amax
    B, SB, gs = gpu_lib.quantize_fp4(_dev(w1), NV)
    q, s, g = fp4.quantize_nv(w1)
    assert np.array_equal(SB.cpu().numpy(), s) and np.array_equal(B.cpu().numpy(), q)
    B, SB, _ = gpu_lib.quantize_fp4(_dev(w1), MX)
    q, s = fp4.quantize_mx(w1)
    assert np.array_equal(SB.cpu().numpy(), s) and np.array_equal(B.cpu().numpy(), q)


def test_every_bf16_value(gpu_lib):
    """Every finite bf16 pattern in a group with every other of its binade and sign, and the special groups."""
    bits = np.arange(65536, dtype=np.uint16).reshape(1, -1, 64)
    for fmt in (MX, NV):
        B, SB, gs = gpu_lib.quantize_fp4(_dev(bits), fmt)
        if fmt == MX:
            q, s = fp4.quantize_mx(bits)
        else:
            q, s, g = fp4.quantize_nv(bits)
            assert np.array_equal(gs.cpu().numpy(), g)
        assert np.array_equal(SB.cpu().numpy(), s) and np.array_equal(B.cpu().numpy(), q)
    x = np.zeros((2, 2, 64), np.uint16)
    x[0, 0, 3] = 0x7F80
    x[0, 1, 40] = 0x7FC0
    x[0, 1, :4] = bf16_rne_bits([6.0, -6.5, 3.0, 2.0 ** -130])
    x[1] = bf16_rne_bits(np.full((2, 64), 2.0 ** -110))   # an expert below the floor of NVFP4's scale
    q, s = fp4.quantize_mx(x)
    B, SB, _ = gpu_lib.quantize_fp4(_dev(x), MX)
    assert np.array_equal(SB.cpu().numpy(), s) and np.array_equal(B.cpu().numpy(), q)
    back = gpu_lib.dequantize_fp4(B, SB, MX).float().cpu()
    assert torch.isnan(back[0, 0, :32]).all() and torch.isnan(back[0, 1, 32:]).all() and torch.isfinite(back[1]).all()
    q, s, g = fp4.quantize_nv(x)
    B, SB, gs = gpu_lib.quantize_fp4(_dev(x), NV)
    assert np.array_equal(SB.cpu().numpy(), s) and np.array_equal(B.cpu().numpy(), q)
    assert np.array_equal(gs.cpu().numpy(), g) and float(gs[1]) == 1.0
    assert torch.isnan(gpu_lib.dequantize_fp4(B, SB, NV, gs).float()[0, 0, :16]).all()


def test_every_scale_code_back(gpu_lib):
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 4))
    q = fp4.pack(codes)
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    for nv, scales in ((False, s[:, :2]), (True, s)):
        want = bf16_rne_bits(fp4.decode_f64(q, scales, nv))
        got = _bits(gpu_lib.dequantize_fp4(torch.from_numpy(q).cuda(), torch.from_numpy(scales.copy()).cuda(), int(nv)))
        nan = np.isnan(bf16_bits_to_f64(want))
        assert np.array_equal(np.isnan(bf16_bits_to_f64(got)), nan) and np.array_equal(got[~nan], want[~nan])


def test_quantised_weights_in_the_products(gpu_lib):
    """What quantize_fp4 writes is what grouped_gemm_a16 reads, in both formats."""
    E, N, K, counts = 3, 64, 256, [5, 0, 9]
    off = torch.tensor([0, 5, 5, 14], dtype=torch.int32).cuda()
    w, a = _weights(E, N, K, 1), bf16_rne_bits(np.random.default_rng(2).standard_normal((14, K)))
    for fmt in (MX, NV):
        B, SB, gs = gpu_lib.quantize_fp4(_dev(w), fmt)
        C = gpu_lib.grouped_gemm_a16(_dev(a), B, SB, fmt, off, expert_scales=gs).double().cpu().numpy()
        q = fp4.quantize_mx(w) if fmt == MX else fp4.quantize_nv(w)
        Wf = fp4.decode_f64(q[0], q[1], fmt == NV, q[2] if fmt == NV else None)
        Af = bf16_bits_to_f64(a)
        want, mag = grouped.forward_f64(Af, Wf, off.cpu().numpy()), grouped.forward_f64(Af, Wf, off.cpu().numpy(), True)
        err = fp32_sum_eps(K) * mag + 2.0 ** -23 * np.abs(want)     # NVFP4: the expert's scale, one more product
        assert np.all(np.abs(C - want) <= err + 2.0 ** -8 * (np.abs(want) + err))


@pytest.mark.parametrize("T,k,K", [(1, 1, 32), (3, 2, 96), (64, 8, 6144), (37, 3, 1056), (5, 8, 16384)])
def test_quantize_gather(gpu_lib, T, k, K):
    rng = np.random.default_rng(T + K)
    ids = rng.integers(0, 12, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    _, off, rows = route_ref(ids, 12)
    R = int(off[-1]) + 3
    x = _weights(1, T, K, 3)[0]
    A = torch.full((R, K // 2), 0x5A, dtype=torch.uint8, device="cuda")
    SA = torch.full((R, K // 32), 0x77, dtype=torch.uint8, device="cuda")
    wA, wS = fp4.gather_mx(x, rows, k, R, A.cpu().numpy(), SA.cpu().numpy())
    gpu_lib.quantize_gather_fp4(_dev(x), torch.from_numpy(rows.astype(np.int32)).cuda(), k, R, A=A, SA=SA)
    assert np.array_equal(A.cpu().numpy(), wA) and np.array_equal(SA.cpu().numpy(), wS)


def _product(gpu_lib, counts, N, K, A, SA, B, SB, eps, extra=2):
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    R = A.shape[0]
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    c = lambda v: torch.from_numpy(v).cuda()
    C = gpu_lib.grouped_gemm_a4(c(A), c(SA), c(B), c(SB), off, out=out)
    Af, Bf, offs = fp4.decode_f64(A, SA, False), fp4.decode_f64(B, SB, False), off.cpu().numpy()
    want, mag = grouped.forward_f64(Af, Bf, offs), grouped.forward_f64(Af, Bf, offs, absolute=True)
    n = sum(counts)
    assert (C[n:] == 7.0).all()
    g = C.double().cpu().numpy()[:n]
    err = fp32_sum_eps(K, eps) * mag[:n]
    assert np.all(np.abs(g - want[:n]) <= err + 2.0 ** -8 * (np.abs(want[:n]) + err) + 2.0 ** -134)
    return C


COUNTS = [([1], 32, 128), ([5, 0, 3], 64, 256), ([64, 1, 63, 65], 128, 640), ([130, 0, 257, 31], 288, 384),
          ([16] * 12, 256, 512), ([300, 700], 544, 1024), ([3, 1, 4] * 30, 64, 128), ([128, 127, 129], 96, 3584),
          # long sums over few tiles, in slices
          ([5, 0, 3], 64, 8192), ([40, 2], 96, 4224), ([1], 32, 2048)]


@pytest.mark.parametrize("counts,N,K", COUNTS)
def test_product(gpu_lib, counts, N, K):
    rng = np.random.default_rng(N + K)
    R, E = sum(counts) + 2, len(counts)
    A, SA = fp4.quantize_mx(bf16_rne_bits(rng.standard_normal((R, K))))
    B, SB = fp4.quantize_mx(bf16_rne_bits(rng.standard_normal((E, N, K)) * 0.02))
    _product(gpu_lib, counts, N, K, A, SA, B, SB, 2.0 ** -16)
    # any codes, scales over 12 binades each
    A, B = (rng.integers(0, 256, v.shape, dtype=np.uint8) for v in (A, B))
    SA, SB = (rng.integers(120, 132, v.shape, dtype=np.uint8) for v in (SA, SB))
    _product(gpu_lib, counts, N, K, A, SA, B, SB, GROUP_EPS_RANDOM_CODES)


def test_product_nan_scales_and_bad_offsets(gpu_lib):
    rng = np.random.default_rng(1)
    counts, N, K = [40, 50], 64, 256
    A, B = rng.integers(0, 256, (90, K // 2), dtype=np.uint8), rng.integers(0, 256, (2, N, K // 2), dtype=np.uint8)
    SA, SB = np.full((90, K // 32), 127, np.uint8), np.full((2, N, K // 32), 127, np.uint8)
    clean = _product(gpu_lib, counts, N, K, A, SA, B, SB, 2.0 ** -16)
    SA[17, 3] = 255
    SB[1, 9, 7] = 255
    c = lambda v: torch.from_numpy(v).cuda()
    off = torch.tensor([0, 40, 90], dtype=torch.int32).cuda()
    C = gpu_lib.grouped_gemm_a4(c(A), c(SA), c(B), c(SB), off)
    nan = torch.zeros((90, N), dtype=torch.bool, device="cuda")
    nan[17] = True
    nan[40:, 9] = True
    assert torch.equal(torch.isnan(C), nan) and torch.equal(C[~nan], clean[~nan])
    for bad in ([1, 40, 90], [0, 50, 40], [0, 40, 91]):
        out = torch.full((90, N), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu_lib.grouped_gemm_a4(c(A), c(SA), c(B), c(SB), torch.tensor(bad, dtype=torch.int32).cuda(), out=out)
        assert (out == 7.0).all()


def test_refusals_and_empty(gpu_lib):
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    gs = torch.ones(2, device="cuda")
    B, SB, _ = gpu_lib.quantize_fp4(x, MX)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: gpu_lib.quantize_fp4(x, 2), lambda: gpu_lib.quantize_fp4(x, MX, expert_scales=gs),
                 lambda: gpu_lib.quantize_fp4(x[:, :, :48].contiguous(), MX),
                 lambda: gpu_lib.quantize_fp4(x[0, 0], MX), lambda: gpu_lib.quantize_fp4(x, MX, B=B[:1]),
                 lambda: gpu_lib.dequantize_fp4(B, SB, NV), lambda: gpu_lib.dequantize_fp4(B, SB, 2),
                 lambda: gpu_lib.grouped_gemm_a4(B[0], SB[0], B, SB[:, :, :1], off),
                 lambda: gpu_lib.grouped_gemm_a4(B[0], SB[0], B, SB, off[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gpu_lib.grouped_gemm_a4(B[0], SB[0], B, SB, off),          # K = 64
                 lambda: gpu_lib.quantize_fp4(x.view(-1)[4:4 + 256].view(1, 4, 64), MX)):   # 8-byte alignment
        with pytest.raises(gpu_lib.W4A8Error):
            call()
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    for fmt in (MX, NV):
        B, SB, g = gpu_lib.quantize_fp4(e, fmt)
        assert B.shape == (0, 32) and gpu_lib.dequantize_fp4(B, SB, fmt, g).shape == (0, 64)
        assert g is None if fmt == MX else (g == 1).all()
    A, SA = gpu_lib.quantize_gather_fp4(e, torch.empty(0, dtype=torch.int32, device="cuda"), 2, 3)
    assert A.shape == (3, 32) and (A == 0).all() and (SA == 0).all()
    Bw, SBw, _ = gpu_lib.quantize_fp4(torch.zeros((2, 32, 128), dtype=torch.bfloat16, device="cuda"), MX)
    empty = torch.empty((0, 64), dtype=torch.uint8, device="cuda"), torch.empty((0, 4), dtype=torch.uint8, device="cuda")
    assert gpu_lib.grouped_gemm_a4(*empty, Bw, SBw, off).shape == (0, 32)


def test_offsets_past_32_bits(gpu_lib):
    E, N, K = 2, 140000, 8192                            # 2.3e9 weights
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[-1, -1] = 3.0
    for fmt in (MX, NV):
        B, SB, gs = gpu_lib.quantize_fp4(w, fmt)
        back = gpu_lib.dequantize_fp4(B, SB, fmt, gs)
        assert (back[-1, -1] == 3.0).all() and (back[-1, -2] == 0).all() and (back[0] == 0).all()
    del w, back
    B, SB, _ = gpu_lib.quantize_fp4(torch.ones((1, 32, 128), dtype=torch.bfloat16, device="cuda"), MX)
    R = 1 << 20
    A = torch.zeros((R, 64), dtype=torch.uint8, device="cuda")
    SA = torch.full((R, 4), 127, dtype=torch.uint8, device="cuda")
    A[-1] = 0x22
    C = gpu_lib.grouped_gemm_a4(A, SA, B, SB, torch.tensor([0, R], dtype=torch.int32).cuda())
    assert (C[-1] == 128).all() and (C[:-1] == 0).all()
