"""Dispatch, its gradient and the combine's gradient on the GPU against
oracle/moves.py: every bf16 result bit for bit, the weights' gradient within
the bound of an fp32 sum of exact products, (N / 64 + 16) 2^-24 of the
products' magnitudes (64 lanes at least, each a chain of N / 64 terms, then
a tree)."""

import numpy as np
import pytest
import torch

from oracle import combine_backward_ref, dispatch_backward_ref, dispatch_ref, route_ref

pytestmark = pytest.mark.gpu


def _bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(torch.bfloat16)


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _routing(T, k, E, seed, drop=0.1):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    if T > 2:
        ids[1] = -1                      # a token without a row
    counts, off, rows = route_ref(ids, E)
    return rows, int(off[-1])


CASES = [(1, 1, 8), (1, 1, 1), (3, 2, 7), (5, 8, 64), (37, 3, 1001), (64, 8, 6144), (17, 10, 520), (9, 1, 8192),
         (33, 17, 4104), (4, 70, 24), (2, 8, 20000)]


@pytest.mark.parametrize("T,k,W", CASES)
def test_dispatch_and_backward(gpu_lib, T, k, W):
    rng = np.random.default_rng(T * 100 + W)
    rows, R = _routing(T, k, 12, W)
    extra = R + 3                                        # rows past the routed ones keep their content
    x, dA = _bf(rng, T, W), _bf(rng, extra, W)
    ros = torch.from_numpy(rows.astype(np.int32)).cuda()
    out = torch.full((extra, W), 7.0, dtype=torch.bfloat16, device="cuda")
    init = _bits(out)
    A = gpu_lib.dispatch(x.cuda(), ros, k, extra, out=out)
    assert np.array_equal(_bits(A), dispatch_ref(_bits(x), rows, k, extra, init))
    dx = gpu_lib.dispatch_backward(dA.cuda(), ros, k)
    assert np.array_equal(_bits(dx), dispatch_backward_ref(_bits(dA), rows, T, k))


@pytest.mark.parametrize("T,k,W", CASES)
def test_combine_backward(gpu_lib, T, k, W):
    rng = np.random.default_rng(T * 100 + W + 1)
    rows, R = _routing(T, k, 12, W + 1)
    extra = R + 2
    C, dout = _bf(rng, extra, W), _bf(rng, T, W)
    w = rng.random(T * k, dtype=np.float32)
    ros = torch.from_numpy(rows.astype(np.int32)).cuda()
    dC = torch.full((extra, W), 7.0, dtype=torch.bfloat16, device="cuda")
    init = _bits(dC)
    got, dw = gpu_lib.combine_backward(C.cuda(), dout.cuda(), ros, torch.from_numpy(w).cuda(), k, dC=dC)
    ref, rdw, mag = combine_backward_ref(_bits(C), _bits(dout), rows, w, T, k, init)
    assert np.array_equal(_bits(got), ref)
    err = np.abs(dw.cpu().numpy() - rdw)
    bound = mag * (W / 64 + 16) * 2.0 ** -24
    print(f"T={T} k={k} N={W}: largest error / bound {(err / np.maximum(bound, 1e-30)).max():.3f}", flush=True)
    assert (err <= bound).all()
    again = gpu_lib.combine_backward(C.cuda(), dout.cuda(), ros, torch.from_numpy(w).cuda(), k)[1]
    assert torch.equal(again, dw)                        # the same bits on every call


def test_rows_out_of_range_masked_nan_and_misaligned(gpu_lib):
    """Rows outside [0, R) move nothing, NaN in rows that no slot names and in
    weights of slots without a row reaches no output, and buffers that are
    only 2-byte aligned give the same bits as aligned ones."""
    rng = np.random.default_rng(4)
    T, k, W, R = 6, 2, 264, 9
    rows = np.array([0, 3, -1, 8, 9, 1, 2, 1 << 30, -7, 4, 5, 6], np.int32)
    nan = float("nan")
    C, dout = _bf(rng, R, W), _bf(rng, T, W)
    C[7] = nan                                           # named by nobody
    w = rng.random(T * k, dtype=np.float32)
    w[(rows < 0) | (rows >= R)] = nan
    ros = torch.from_numpy(rows).cuda()
    shift = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)]).cuda()[1:].view(t.shape)  # noqa: E731
    for move in (lambda t: t.cuda(), shift):
        dC, dw = gpu_lib.combine_backward(move(C), move(dout), ros, torch.from_numpy(w).cuda(), k)
        ref, rdw, mag = combine_backward_ref(_bits(C), _bits(dout), rows, w, T, k)
        assert np.array_equal(_bits(dC), ref)
        assert (np.abs(dw.cpu().numpy() - rdw) <= mag * (W / 64 + 16) * 2.0 ** -24).all()
        A = gpu_lib.dispatch(move(dout), ros, k, R)
        assert np.array_equal(_bits(A), dispatch_ref(_bits(dout), rows, k, R))
        dx = gpu_lib.dispatch_backward(move(C), ros, k)
        assert np.array_equal(_bits(dx), dispatch_backward_ref(_bits(C), rows, T, k))


def test_gradient_of_combine_against_differences(gpu_lib):
    """<out(w + h v) - out(w - h v), dout> / 2h against <dw, v>, and the same
    in C, with values whose products and sums are exact in bf16."""
    rng = np.random.default_rng(5)
    T, k, N = 4, 3, 64
    rows = torch.from_numpy(rng.permutation(T * k).astype(np.int32)).cuda()
    small = lambda *s: torch.from_numpy(rng.integers(-2, 3, s).astype(np.float32))  # noqa: E731
    C, dout, w = small(T * k, N), small(T, N), small(T * k)
    v, V = small(T * k), small(T * k, N)
    f = lambda c, u: (gpu_lib.combine(c.to(torch.bfloat16).cuda(), rows, u.cuda(), k).double().cpu()  # noqa: E731
                      * dout.double()).sum()
    dC, dw = gpu_lib.combine_backward(C.to(torch.bfloat16).cuda(), dout.to(torch.bfloat16).cuda(), rows, w.cuda(), k)
    assert (f(C, w + v) - f(C, w - v)) / 2 == (dw.cpu().double() * v).sum()
    assert (f(C + V, w) - f(C - V, w)) / 2 == (dC.double().cpu() * V).sum()


def test_moves_offsets_past_32_bits(gpu_lib):
    """A row whose byte offset is past 2^32: the last of 270000 rows of 8192 columns."""
    R, K = 270000, 8192
    big = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((1, K), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    ros = torch.tensor([R - 1], dtype=torch.int32, device="cuda")
    big[R - 1] = 0
    gpu_lib.dispatch(x, ros, 1, R, out=big)
    assert torch.equal(big[R - 1:], x)
    assert torch.equal(gpu_lib.dispatch_backward(big, ros, 1), x)
    one = torch.ones(1, device="cuda")
    dC, dw = gpu_lib.combine_backward(big, x, ros, one, 1, dC=big)
    ref = (x.double() ** 2).sum()
    assert torch.equal(big[R - 1:], x) and abs(dw.double() - ref) < ref * (K / 64 + 16) * 2.0 ** -24


def test_moves_empty_stream_and_refusals(gpu_lib):
    x = torch.ones((3, 16), dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert gpu_lib.dispatch(x[:0], none, 2, 0).shape == (0, 16)
    assert gpu_lib.dispatch_backward(x, none, 2).shape == (0, 16)
    dC, dw = gpu_lib.combine_backward(x, x[:0], none, torch.zeros(0, device="cuda"), 2)
    assert not dC.any() and dw.numel() == 0
    # no rows at all: zeros, nothing read
    ros = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    assert not gpu_lib.dispatch_backward(x[:0], ros, 2).any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = torch.arange(3, dtype=torch.int32, device="cuda")
        a = gpu_lib.dispatch(x * 2, r, 1, 3)
    side.synchronize()
    assert torch.equal(a, x * 2)
    with pytest.raises(ValueError):
        gpu_lib.dispatch(x, ros, 1, 3)                          # 6 slots for 3 tokens of one
    with pytest.raises(ValueError):
        gpu_lib.dispatch_backward(x, ros, 4)
    with pytest.raises(TypeError):
        gpu_lib.dispatch(x.float(), ros, 2, 3)
    with pytest.raises(ValueError):
        gpu_lib.combine_backward(x, x[:, :8], ros, torch.zeros(6, device="cuda"), 2)
    with pytest.raises(ValueError):
        gpu_lib.dispatch(x.t(), torch.zeros(16, dtype=torch.int32, device="cuda"), 1, 3)
