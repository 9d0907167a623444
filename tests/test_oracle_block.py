"""Pins for the oracles of the operators around the expert products
(oracle/gate.py, moves.py, matvec.py, swiglu8.py): closed forms, torch's
autograd in fp64, central differences, and the moves as adjoints of each
other on exact sums."""

import numpy as np
import pytest
import torch

from oracle import (checkpoint_ref, combine_backward_ref, decode_f64, dispatch_backward_ref, dispatch_ref,
                    matvec_f64, swiglu_backward_f64, topk_gate_backward_f64, topk_gate_f64)
from oracle.gate import weights
from oracle.quant import bf16_bits_to_f32

MODES = [(0, False), (0, True), (1, False), (1, True)]


def _bits(x):
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def test_selection_order_ties_and_closed_experts():
    inf, nan = np.inf, np.nan
    l = np.array([[1.0, 3.0, 3.0, -inf, 0.0], [-inf] * 5, [-inf, -inf, 2.0, -inf, -inf],
                  [0.0, -0.0, nan, inf, 1.0], [-3.4e38, -inf, -3.4e38, -inf, -inf]])
    ids, w = topk_gate_f64(l, 3, 0, True)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [2, -1, -1], [2, 3, 4], [0, 2, -1]]
    assert w[1].tolist() == [0, 0, 0] and w[2].tolist() == [1, 0, 0] and np.isnan(w[3]).all()
    assert np.allclose(w[4], [0.5, 0.5, 0.0])
    ids, w = topk_gate_f64(l, 5, 1, False)
    assert ids[3].tolist() == [2, 3, 4, 0, 1] and w[3, 1] == 1.0 and w[3, 3] == 0.5 and np.isnan(w[3, 0])


@pytest.mark.parametrize("score,renorm", MODES)
def test_gate_against_torch_autograd(score, renorm):
    rng = np.random.default_rng(5)
    l = rng.standard_normal((6, 11)) * 2
    l[2, 3] = -np.inf
    ids, w = topk_gate_f64(l, 4, score, renorm, 1.7)
    t = torch.tensor(l, requires_grad=True)
    i = torch.tensor(ids.astype(np.int64))
    p = torch.softmax(t, 1) if score == 0 else torch.sigmoid(t)
    v = p.gather(1, i)
    if renorm:
        v = v / v.sum(1, keepdim=True)
    v = v * 1.7
    assert np.allclose(w, v.detach().numpy(), rtol=1e-12)
    dw = rng.standard_normal(w.shape)
    (v * torch.tensor(dw)).sum().backward()
    d = topk_gate_backward_f64(l, ids, dw, score, renorm, 1.7)
    assert np.allclose(d, t.grad.numpy(), rtol=1e-10, atol=1e-13)


@pytest.mark.parametrize("score,renorm", MODES)
def test_gate_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(6)
    l = rng.standard_normal((3, 7))
    ids, w = topk_gate_f64(l, 3, score, renorm)
    dw = rng.standard_normal(w.shape)
    d = topk_gate_backward_f64(l, ids, dw, score, renorm)
    h = 1e-5
    for t in range(3):
        for e in range(7):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            num = ((weights(a, ids, score, renorm) - weights(b, ids, score, renorm)) * dw).sum() / (2 * h)
            assert abs(num - d[t, e]) < 1e-8


def test_moves_are_adjoint_and_exact():
    rng = np.random.default_rng(7)
    T, k, N, R = 9, 3, 13, 30
    rows = rng.permutation(R)[:T * k].astype(np.int32)
    rows[[4, 11]] = -1, R
    x = _bits(rng.integers(-8, 9, (T, N)))
    dA = _bits(rng.integers(-8, 9, (R, N)))
    A = dispatch_ref(x, rows, k, R)
    dx = dispatch_backward_ref(dA, rows, T, k)
    f = bf16_bits_to_f32
    assert (f(A) * f(dA)).sum() == (f(x) * f(dx)).sum()          # <S x, dA> = <x, S^T dA>, small integers: exact
    w = np.exp2(rng.integers(-2, 3, T * k)).astype(np.float32)
    C = _bits(rng.integers(-8, 9, (R, N)))
    dout = _bits(rng.integers(-8, 9, (T, N)))
    dC, dw, mag = combine_backward_ref(C, dout, rows, w, T, k)
    # out = sum w C is linear in C and in w: <out, dout> = <C, dC> = <w, dw>
    assert (f(C) * f(dC)).sum() == float((w * dw).sum())
    assert dw[4] == dw[11] == 0 and (mag >= np.abs(dw)).all()


def test_matvec_against_loops_and_formats():
    rng = np.random.default_rng(8)
    E, N, K = 3, 5, 64
    x = _bits(rng.standard_normal((2, K)))
    B = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    sc = _bits(rng.random((E, N, K // 32)))
    z = rng.integers(0, 16, (E, N, K // 32)).astype(np.uint8)
    ids = np.array([2, 0, -1, 1], np.int32)
    y, mag = matvec_f64(x, B, sc, 2, ids=ids, zeros=z)
    xf, sf = bf16_bits_to_f32(x).astype(float), bf16_bits_to_f32(sc).astype(float)
    for s, e in enumerate(ids):
        for n in range(N):
            v = 0.0
            for kk in range(K):
                q = (int(B[e, n, kk // 2]) >> (4 * (kk % 2))) & 15
                v += xf[s // 2, kk] * (q - int(z[e, n, kk // 32])) * sf[e, n, kk // 32] if e >= 0 else 0.0
            assert abs(v - y[s, n]) < 1e-10
    assert (mag >= np.abs(y)).all()
    # unit scales: MXFP4 code 127 and NVFP4 code 0x38 are both 1
    a, _ = matvec_f64(x, B[:1], np.full((1, N, K // 32), 127, np.uint8), 0)
    b, _ = matvec_f64(x, B[:1], np.full((1, N, K // 16), 0x38, np.uint8), 1)
    assert np.array_equal(a, b)
    # no zeros given = zeros of 8
    c, _ = matvec_f64(x, B, sc, 2, ids=ids)
    d, _ = matvec_f64(x, B, sc, 2, ids=ids, zeros=np.full_like(z, 8))
    assert np.array_equal(c, d) and not np.array_equal(c, y)


def test_checkpoint_copy():
    rng = np.random.default_rng(9)
    C = _bits(rng.standard_normal((4, 256)) * 3)
    C[1, :128] = 0
    C[2, 128:] = _bits(np.full(128, 2.0 ** -101))
    codes, s = checkpoint_ref(C)
    x = bf16_bits_to_f32(C).astype(float)
    v = decode_f64(codes, s)
    assert s[1, 0] == 1 and s[2, 1] == 1 and not (codes[1, :128] & 0x7F).any() and not codes[2, 128:].any()
    amax = np.abs(x.reshape(4, 2, 128)).max(2).repeat(128).reshape(4, 256)
    # half a step of the value's binade, or of the subnormal grid; 2^-100 for what is dropped
    assert (np.abs(v - x) <= np.maximum(np.abs(x) * 2.0 ** -4, amax / 448 * 2.0 ** -10) * 1.0001 + 2.0 ** -100).all()
    top = np.abs(x) == amax
    assert (codes[top & (amax > 2.0 ** -99)] & 0x7F == 0x7E).all()


def test_swiglu_gradient_against_autograd_and_differences():
    rng = np.random.default_rng(10)
    codes, s = checkpoint_ref(_bits(rng.standard_normal((3, 256)) * 4))
    dh = rng.standard_normal((3, 128))
    dC, h = swiglu_backward_f64(codes, s, dh)
    t = torch.tensor(decode_f64(codes, s), requires_grad=True)
    y = torch.nn.functional.silu(t[:, :128]) * t[:, 128:]
    assert np.allclose(h, y.detach().numpy(), rtol=1e-13)
    (y * torch.tensor(dh)).sum().backward()
    assert np.allclose(dC, t.grad.numpy(), rtol=1e-11, atol=1e-13)
    v = decode_f64(codes, s)

    def f(a):
        g, u = a[:, :128], a[:, 128:]
        return (g / (1 + np.exp(-g)) * u * dh).sum()
    for c in (0, 77, 128, 250):
        a, b = v.copy(), v.copy()
        a[1, c] += 1e-5
        b[1, c] -= 1e-5
        assert abs((f(a) - f(b)) / 2e-5 - dC[1, c]) < 1e-7
