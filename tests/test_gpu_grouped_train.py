"""The grouped products with bf16 weights and their gradients on the GPU
against oracle/grouped.py.

Bound: products of bf16 values are exact in fp32, and a sum of Z of them in
any order, each addition off by an fp32 unit at most, is within (Z + 8) 2^-23 of
the magnitudes' sum; then the output's rounding (bf16 2^-8, fp32 2^-24)."""

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, bf16_rne_bits, grouped

pytestmark = pytest.mark.gpu


def _dev(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def _draw(seed, *shape):
    b = bf16_rne_bits(np.random.default_rng(seed).standard_normal(shape))
    return b, bf16_bits_to_f64(b)


def _off(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


def _check(got, want, mag, Z, half=2.0 ** -8):
    g = got.double().cpu().numpy()
    live = ~np.isnan(want)
    err = (Z + 8) * 2.0 ** -23 * mag
    bound = err + half * (np.abs(want) + err) + 2.0 ** -134
    assert np.all(np.isfinite(g[live]))
    worst = np.max((np.abs(g - want) / bound)[live]) if live.any() else 0.0
    assert worst <= 1.0, worst
    return live


# counts per expert, N, K
CASES = [
    ([1], 8, 8), ([5, 0, 3], 16, 8), ([0, 0, 7], 40, 24), ([64, 1, 63, 65], 128, 96), ([130, 0, 257, 31, 2], 264, 72),
    ([16] * 12, 256, 512), ([128, 127, 129], 520, 136), ([300, 900], 384, 1024), ([3, 1, 4, 1, 5] * 30, 64, 64),
    ([1700, 0, 900], 264, 200), ([2000], 520, 328), ([801, 815], 72, 456),
    # not whole 16-byte pieces
    ([1], 1, 1), ([3, 0, 5], 7, 5), ([40, 33], 33, 31), ([129, 1], 130, 257), ([20, 200], 255, 64), ([65], 64, 129),
    ([1] * 100, 12, 10), ([40, 3], 132, 64), ([200, 90], 388, 72),
]
# long sums over few tiles, taken in slices (of K, of N or of the rows); ends inside and at the start of a slice
LONG = [
    ([3, 0, 7], 72, 5000), ([2], 128, 5969), ([40, 1], 4352, 64), ([9, 0, 60], 4097, 33), ([6000, 0, 30], 40, 24),
    ([5, 5000], 31, 17), ([1, 1], 16, 1024), ([30, 0], 1024, 1024), ([513, 1023, 0, 2048], 64, 8),
]


def test_long_sums_are_sliced(gpu_lib):
    need = gpu_lib.load().w4a8_grouped_gemm_workspace_bytes
    for counts, N, K in LONG:
        assert any(need(product, sum(counts), len(counts), N, K) for product in (0, 1, 2))


@pytest.mark.parametrize("counts,N,K", CASES + LONG)
def test_forward_and_gradients(gpu_lib, counts, N, K):
    R, E, extra = sum(counts), len(counts), 3
    A, Af = _draw(N + K, R + extra, K)
    W, Wf = _draw(N + K + 1, E, N, K)
    dC, dCf = _draw(N + K + 2, R + extra, N)
    A[R:] = 0x7FC0                                      # rows behind the last expert hold NaN and are not touched
    dC[R:] = 0x7F80
    off, Ad, Wd, dCd = _off(counts), _dev(A), _dev(W), _dev(dC)
    offs = off.cpu().numpy()
    for name, args, ref, Z, width in (("grouped_gemm_bf16", (Ad, Wd), (grouped.forward_f64, Af, Wf), K, N),
                                      ("grouped_gemm_dgrad", (dCd, Wd), (grouped.dgrad_f64, dCf, Wf), N, K)):
        out = torch.full((R + extra, width), 7.0, dtype=torch.bfloat16, device="cuda")
        got = getattr(gpu_lib, name)(*args, off, out=out)
        _check(got, ref[0](*ref[1:], offs), ref[0](*ref[1:], offs, absolute=True), Z)
        assert (got[R:] == 7.0).all()
        assert torch.equal(getattr(gpu_lib, name)(*args, off)[:R], got[:R])
    want, mag = grouped.wgrad_f64(dCf, Af, offs), grouped.wgrad_f64(dCf, Af, offs, absolute=True)
    got = gpu_lib.grouped_gemm_wgrad(dCd, Ad, off)
    assert got.dtype == torch.float32 and got.shape == (E, N, K)
    _check(got, want, mag, max(counts), 2.0 ** -24)
    out16 = torch.full((E, N, K), 5.0, dtype=torch.bfloat16, device="cuda")
    _check(gpu_lib.grouped_gemm_wgrad(dCd, Ad, off, out=out16), want, mag, max(counts))
    # accumulation: one more addition and, in bf16, one rounding of the new sum
    base = _draw(9, E, N, K)[0]
    for t, half in ((_dev(base), 2.0 ** -8), (_dev(base).float(), 2.0 ** -24)):
        b = t.double().cpu().numpy()
        gpu_lib.grouped_gemm_wgrad(dCd, Ad, off, out=t, accumulate=True)
        _check(t, want + b, mag + np.abs(b), max(counts) + 1, half)
        idle = [e for e, c in enumerate(counts) if c == 0]
        assert np.array_equal(t.double().cpu().numpy()[idle], b[idle])


@pytest.mark.parametrize("shift", [1, 4])
def test_unaligned_buffers(gpu_lib, shift):
    counts, N, K = [70, 0, 30], 72, 64
    off = _off(counts)
    A, W, dC = (_dev(_draw(i, *s)[0]) for i, s in enumerate([(100, K), (3, N, K), (100, N)]))

    def moved(t):
        b = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        v = b[shift:shift + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    for f, a, b in ((gpu_lib.grouped_gemm_bf16, A, W), (gpu_lib.grouped_gemm_dgrad, dC, W),
                    (gpu_lib.grouped_gemm_wgrad, dC, A)):
        want = f(a, b, off).float()
        for x, y in ((moved(a), b), (a, moved(b)), (moved(a), moved(b))):
            assert torch.allclose(f(x, y, off).float(), want, rtol=2.0 ** -7, atol=1e-4)
        o = moved(torch.zeros_like(f(a, b, off)))
        assert torch.allclose(f(a, b, off, out=o).float(), want, rtol=2.0 ** -7, atol=1e-4)


def test_neighbours_stay_out(gpu_lib):
    """Infinities and NaN of one expert's rows and weights do not reach another's results."""
    counts, N, K = [33, 47, 20], 64, 72
    off = _off(counts)
    A, W, dC = _draw(1, 100, K)[0], _draw(2, 3, N, K)[0], _draw(3, 100, N)[0]
    clean = [gpu_lib.grouped_gemm_bf16(_dev(A), _dev(W), off), gpu_lib.grouped_gemm_dgrad(_dev(dC), _dev(W), off),
             gpu_lib.grouped_gemm_wgrad(_dev(dC), _dev(A), off)]
    A[33:80] = 0x7F80
    dC[33:80] = 0x7FC0
    W[1] = 0xFF80
    got = [gpu_lib.grouped_gemm_bf16(_dev(A), _dev(W), off), gpu_lib.grouped_gemm_dgrad(_dev(dC), _dev(W), off),
           gpu_lib.grouped_gemm_wgrad(_dev(dC), _dev(A), off)]
    for c, g in zip(clean[:2], got[:2]):
        assert torch.equal(g[:33], c[:33]) and torch.equal(g[80:], c[80:]) and not torch.isfinite(g[33:80]).any()
    assert torch.equal(got[2][0], clean[2][0]) and torch.equal(got[2][2], clean[2][2])
    assert torch.isnan(got[2][1]).all()


@pytest.mark.parametrize("bad", [[1, 4, 8], [0, 5, 4], [0, 4, 9], [-1, 4, 8]])
def test_bad_offsets_write_nothing(gpu_lib, bad):
    off = torch.tensor(bad, dtype=torch.int32).cuda()
    A, W, dC = (_dev(_draw(i, *s)[0]) for i, s in enumerate([(8, 16), (2, 24, 16), (8, 24)]))
    o = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in ((8, 24), (8, 16), (2, 24, 16))]
    gpu_lib.grouped_gemm_bf16(A, W, off, out=o[0])
    gpu_lib.grouped_gemm_dgrad(dC, W, off, out=o[1])
    gpu_lib.grouped_gemm_wgrad(dC, A, off, out=o[2])
    assert all((t == 7.0).all() for t in o)


@pytest.mark.parametrize("bad", [[1, 4, 8], [0, 5, 4], [0, 4, 9], [-1, 4, 8]])
def test_bad_offsets_write_nothing_in_slices(gpu_lib, bad):
    off = torch.tensor(bad, dtype=torch.int32).cuda()
    A, W, V, dC = (_dev(_draw(i, *s)[0]) for i, s in enumerate([(8, 1024), (2, 24, 1024), (2, 1024, 16), (8, 1024)]))
    o = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in ((8, 24), (8, 16))]
    gpu_lib.grouped_gemm_bf16(A, W, off, out=o[0])
    gpu_lib.grouped_gemm_dgrad(dC, V, off, out=o[1])
    off = (off * 256).contiguous()
    A, dC = (_dev(_draw(i, *s)[0]) for i, s in enumerate([(2048, 16), (2048, 24)]))
    o.append(torch.full((2, 24, 16), 7.0, dtype=torch.bfloat16, device="cuda"))
    gpu_lib.grouped_gemm_wgrad(dC, A, off, out=o[2])
    assert all((t == 7.0).all() for t in o)


def test_without_a_workspace(gpu_lib):
    """NULL: the sum in one piece; the same within the sums' bound."""
    lib, R, E, N, K = gpu_lib.load(), 10, 3, 72, 5000
    (A, Af), (W, Wf) = _draw(1, R, K), _draw(2, E, N, K)
    off, Ad, Wd = _off([3, 0, 7]), _dev(A), _dev(W)
    out = torch.empty((R, N), dtype=torch.bfloat16, device="cuda")
    assert lib.w4a8_grouped_gemm_bf16(Ad.data_ptr(), Wd.data_ptr(), off.data_ptr(), R, E, N, K, out.data_ptr(), None, 0,
                                      torch.cuda.current_stream().cuda_stream) == 0
    offs = off.cpu().numpy()
    _check(out, grouped.forward_f64(Af, Wf, offs), grouped.forward_f64(Af, Wf, offs, absolute=True), K)


def test_slices_on_two_streams_and_in_graphs(gpu_lib):
    """Calls that may run at a time have workspaces of their own; replays give the eager results."""
    off = _off([3, 0, 7])
    A, W = [_dev(_draw(i, 10, 5000)[0]) for i in range(2)], _dev(_draw(7, 3, 72, 5000)[0])
    want = [gpu_lib.grouped_gemm_bf16(a, W, off) for a in A]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in A]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(gpu_lib.grouped_gemm_bf16(A[i], W, off))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
    graphs, outs = [], []
    for a in A:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(gpu_lib.grouped_gemm_bf16(a, W, off))
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert torch.equal(gpu_lib.grouped_gemm_bf16(A[0], W, off), want[0])


def test_many_experts(gpu_lib):
    rng = np.random.default_rng(11)
    counts = rng.integers(0, 4, 2048)
    R, N, K = int(counts.sum()), 16, 40
    off = _off(counts)
    offs = off.cpu().numpy()
    (A, Af), (W, Wf), (dC, dCf) = _draw(1, R, K), _draw(2, 2048, N, K), _draw(3, R, N)
    _check(gpu_lib.grouped_gemm_bf16(_dev(A), _dev(W), off), grouped.forward_f64(Af, Wf, offs),
           grouped.forward_f64(Af, Wf, offs, absolute=True), K)
    _check(gpu_lib.grouped_gemm_dgrad(_dev(dC), _dev(W), off), grouped.dgrad_f64(dCf, Wf, offs),
           grouped.dgrad_f64(dCf, Wf, offs, absolute=True), N)
    _check(gpu_lib.grouped_gemm_wgrad(_dev(dC), _dev(A), off), grouped.wgrad_f64(dCf, Af, offs),
           grouped.wgrad_f64(dCf, Af, offs, absolute=True), 4, 2.0 ** -24)


def test_gradients_by_differences(gpu_lib):
    """The GPU's gradients along one direction against differences of the oracle's forward pass (exact in fp64:
    the product is linear in each operand)."""
    counts, N, K = [20, 13], 48, 40
    off = _off(counts)
    offs = off.cpu().numpy()
    (A, Af), (W, Wf), (dC, dCf) = _draw(1, 33, K), _draw(2, 2, N, K), _draw(3, 33, N)
    dA = gpu_lib.grouped_gemm_dgrad(_dev(dC), _dev(W), off).double().cpu().numpy()
    dW = gpu_lib.grouped_gemm_wgrad(_dev(dC), _dev(A), off).double().cpu().numpy()
    f = lambda a, w: float(np.sum(grouped.forward_f64(a, w, offs) * dCf))
    rng = np.random.default_rng(4)
    u, v = rng.standard_normal(Af.shape), rng.standard_normal(Wf.shape)
    ma = np.sum(np.abs(u) * grouped.dgrad_f64(dCf, Wf, offs, absolute=True))
    mw = np.sum(np.abs(v) * grouped.wgrad_f64(dCf, Af, offs, absolute=True))
    assert abs(np.sum(u * dA) - (f(Af + u, Wf) - f(Af - u, Wf)) / 2) <= 2.0 ** -8 * np.sum(np.abs(u * dA)) + (
        N + 8) * 2.0 ** -22 * ma
    assert abs(np.sum(v * dW) - (f(Af, Wf + v) - f(Af, Wf - v)) / 2) <= 2.0 ** -24 * np.sum(np.abs(v * dW)) + (
        20 + 8) * 2.0 ** -22 * mw


def test_empty_and_refusals(gpu_lib):
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    A0, W = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"), _dev(_draw(1, 2, 24, 16)[0])
    assert gpu_lib.grouped_gemm_bf16(A0, W, z).shape == (0, 24)
    d0 = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.grouped_gemm_dgrad(d0, W, z).shape == (0, 16)
    assert (gpu_lib.grouped_gemm_wgrad(d0, A0, z, out=torch.full((2, 24, 16), 7.0, device="cuda")) == 0).all()
    A = _dev(_draw(2, 8, 16)[0])
    for call in (lambda: gpu_lib.grouped_gemm_bf16(A, W, z[:2]), lambda: gpu_lib.grouped_gemm_dgrad(A, W, z),
                 lambda: gpu_lib.grouped_gemm_bf16(A.t(), W, z), lambda: gpu_lib.grouped_gemm_wgrad(A, d0, z),
                 lambda: gpu_lib.grouped_gemm_wgrad(A, A, z, accumulate=True),
                 lambda: gpu_lib.grouped_gemm_bf16(A, W, z, out=torch.empty((8, 23), dtype=torch.bfloat16, device="cuda")),
                 lambda: gpu_lib.grouped_gemm_bf16(A.cpu(), W, z)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gpu_lib.grouped_gemm_bf16(A.float(), W, z), lambda: gpu_lib.grouped_gemm_bf16(A, W, z.long()),
                 lambda: gpu_lib.grouped_gemm_wgrad(A, A, z, out=[0.0]),
                 lambda: gpu_lib.grouped_gemm_wgrad(A, A, z, out=torch.empty((2, 16, 16), dtype=torch.float16, device="cuda"))):
        with pytest.raises(TypeError):
            call()


def test_wide_weights(gpu_lib):
    """More columns than a tile's 32-bit offsets span."""
    N, K = (1 << 22) + 8, 8
    off = _off([2, 3])
    A, W = _draw(1, 5, K)[0], torch.zeros((2, N, K), dtype=torch.bfloat16, device="cuda")
    W[1, -3:] = 1.0
    C = gpu_lib.grouped_gemm_bf16(_dev(A), W, off)
    want = bf16_bits_to_f64(A)[2:].sum(axis=1)
    assert np.allclose(C[2:, -3:].double().cpu().numpy(), want[:, None], rtol=2.0 ** -7, atol=2.0 ** -7)
    assert (C[:, :-3] == 0).all() and (C[:2] == 0).all()
    dA = gpu_lib.grouped_gemm_dgrad(torch.ones_like(C), W, off)
    assert (dA[2:] == 3.0).all() and (dA[:2] == 0).all()
    dW = gpu_lib.grouped_gemm_wgrad(C, _dev(A), off, out=W)
    assert (dW[0] == 0).all() and (dW[1, :-3] == 0).all() and (dW[1, -3:] != 0).any()


def test_offsets_past_32_bits(gpu_lib):
    N, K, E = 8192, 8, 2
    R = 270000                                          # R * N = 2.2e9
    off = torch.tensor([0, R - 5, R], dtype=torch.int32).cuda()
    A = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    A[-5:] = 1.0
    W = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    W[1, :, 0] = torch.arange(N, device="cuda") % 128
    C = gpu_lib.grouped_gemm_bf16(A, W, off)
    assert torch.equal(C[-5:], W[1, :, 0].expand(5, N)) and (C[:1000] == 0).all() and (C[-1000:-5] == 0).all()
    C[-5:] = 2.0
    dA = gpu_lib.grouped_gemm_dgrad(C, W, off)
    assert (dA[-5:, 0].float() == float(2 * W[1, :, 0].double().sum())).all() and (dA[:-5] == 0).all()
    del C, dA
    E, N, K = 40, 8192, 8192                            # E * N * K = 2.7e9
    W = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    W[-1, -1] = 1.0
    A = torch.ones((3, K), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0] * E + [3], dtype=torch.int32).cuda()
    C = gpu_lib.grouped_gemm_bf16(A, W, off)
    assert (C[:, -1] == K).all() and (C[:, :-1] == 0).all()
    dW = gpu_lib.grouped_gemm_wgrad(C, A, off, out=W)
    assert (dW[-1, -1] == 3 * K).all() and (dW[-1, :-1] == 0).all() and (dW[0] == 0).all()
