"""Pins of the oracles of the norm, the 4-bit quantiser, the grouped products'
gradients and the clipping: closed forms, torch's autograd in fp64, central
differences, exact rationals."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, bf16_rne_bits, e4m3_table, fp4, grouped, norm


def _bits(rng, *shape, scale=1.0):
    return bf16_rne_bits(rng.standard_normal(shape) * scale)


def test_norm_closed_forms():
    ones = np.full((1, 8), 0x3F80, np.uint16)
    assert np.allclose(norm.rms_norm_f64(ones, None, 0.0), 1.0)
    assert np.allclose(norm.rms_norm_f64(ones, np.arange(8.0), 3.0), np.arange(8.0) / 2)
    x = _bits(np.random.default_rng(0), 3, 40)
    y = norm.rms_norm_f64(x, None, 0.0)
    assert np.allclose(np.mean(y * y, axis=1), 1.0)
    assert np.array_equal(norm.rms_norm_f64(bf16_rne_bits(4 * bf16_bits_to_f64(x)), None, 0.0), y)   # scale drops out


def test_norm_sum_is_torchs():
    rng = np.random.default_rng(1)
    a, b = _bits(rng, 5, 64), _bits(rng, 5, 64, scale=1000.0)
    t = lambda v: torch.from_numpy(v.view(np.int16).copy()).view(torch.bfloat16)
    want = (t(a).float() + t(b).float()).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(norm.sum_bits(a, b), want)


@pytest.mark.parametrize("with_w,with_r", [(True, False), (False, True)])
def test_norm_backward_autograd_and_differences(with_w, with_r):
    rng = np.random.default_rng(2)
    h, dy, r = _bits(rng, 4, 24), _bits(rng, 4, 24), _bits(rng, 4, 24)
    w = rng.standard_normal(24) if with_w else None
    dx, dw, _, _ = norm.rms_norm_backward_f64(h, w, dy, 1e-3, r if with_r else None)
    H = torch.tensor(bf16_bits_to_f64(h), requires_grad=True)
    W = torch.tensor(w if with_w else np.ones(24), requires_grad=True)
    y = H / torch.sqrt((H * H).mean(1, keepdim=True) + float(np.float32(1e-3))) * W
    G = torch.tensor(bf16_bits_to_f64(dy))
    loss = (y * G).sum() + ((H * torch.tensor(bf16_bits_to_f64(r))).sum() if with_r else 0)
    loss.backward()
    assert np.allclose(dx, H.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(dw, W.grad.numpy(), rtol=1e-12, atol=1e-14)
    # along one direction, by differences of the forward definition
    d = rng.standard_normal((4, 24))
    f = lambda H_: float(np.sum(H_ / np.sqrt(np.mean(H_ * H_, axis=1, keepdims=True) + float(np.float32(1e-3)))
                                * (1.0 if w is None else w) * bf16_bits_to_f64(dy)))
    H0 = bf16_bits_to_f64(h)
    diff = (f(H0 + 1e-6 * d) - f(H0 - 1e-6 * d)) / 2e-6
    own = float(np.sum(d * (dx - (bf16_bits_to_f64(r) if with_r else 0))))
    assert abs(diff - own) < 1e-7 * max(1.0, abs(own))


def test_e4m3_nearest_is_torchs():
    rng = np.random.default_rng(3)
    v = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.integers(-4, 3, 20000), e4m3_table()[:127],
                        (e4m3_table()[1:127] + e4m3_table()[:126]) / 2]).clip(-448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(norm.e4m3_nearest(v), want.astype(np.float64))


def test_check_codes_rejects_mistakes():
    rng = np.random.default_rng(4)
    y = rng.standard_normal((3, 256))
    s = np.abs(y.reshape(3, 2, 128)).max(axis=2) / 448
    grid = {v: c for c, v in enumerate(e4m3_table()) if np.isfinite(v)}
    q = norm.e4m3_nearest(y.reshape(3, 2, 128) / s[:, :, None])
    codes = np.array([grid[v] for v in q.ravel()], np.uint8).reshape(3, 256)
    assert norm.check_codes(codes, s, y, 0.0) == 0
    bad = codes.copy()
    bad[1, 7] ^= 1
    assert norm.check_codes(bad, s, y, 2.0 ** -20) == 1
    assert norm.check_codes(codes, s * (1 + 2.0 ** -16), y, 2.0 ** -20) >= 6
    assert norm.check_codes(codes, s, np.roll(y, 1, axis=1), 2.0 ** -20) > 100


GRID = [Fraction(v) for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]


def _frac_code(x, scale):
    q = abs(Fraction(x)) / scale
    best = min(range(8), key=lambda i: (abs(GRID[i] - q), i % 2)) if q < 6 else 7
    return best | (8 if np.signbit(x) else 0)


def test_fp4_against_rationals():
    rng = np.random.default_rng(5)
    x = bf16_rne_bits(rng.standard_normal((2, 3, 64)) * 0.02)
    x[0, 0, :8] = bf16_rne_bits([0.0, -0.0, 1.0, 0.25, 0.125, 0.1875, -0.75, 0.875])   # ties at scale 2^-2
    v = bf16_bits_to_f64(x)
    q, s = fp4.quantize_mx(x)
    codes = fp4.unpack(q)
    for idx in np.ndindex(2, 3, 2):
        blk = v[idx[0], idx[1], 32 * idx[2]:32 * idx[2] + 32]
        e = 0
        a = max(abs(Fraction(t)) for t in blk)
        while Fraction(2) ** (e + 3) <= a:
            e += 1
        while Fraction(2) ** (e + 2) > a:
            e -= 1
        assert s[idx] == e + 127
        assert [int(c) for c in codes[idx[0], idx[1], 32 * idx[2]:32 * idx[2] + 32]] == [
            _frac_code(t, Fraction(2) ** e) for t in blk]
    q, s, gs = fp4.quantize_nv(x)
    codes, e4 = fp4.unpack(q), [Fraction(t) for t in e4m3_table()[:127]]
    for e in range(2):
        top = np.abs(v[e]).max()
        assert gs[e] == np.float32(np.float32(top) / np.float32(2688))
        g = Fraction(float(gs[e]))
        for n, b in np.ndindex(3, 4):
            blk = v[e, n, 16 * b:16 * b + 16]
            r = max(abs(Fraction(t)) for t in blk) / (6 * g)
            sc = min(range(127), key=lambda i: (abs(e4[i] - r), i % 2))
            assert s[e, n, b] == sc
            if sc:
                assert [int(c) for c in codes[e, n, 16 * b:16 * b + 16]] == [_frac_code(t, e4[sc] * g) for t in blk]


def test_fp4_special_groups():
    x = np.zeros((1, 2, 64), np.uint16)
    x[0, 0, 3] = 0x7F80                    # an infinity, alone among zeros
    x[0, 1, 40] = 0x7FC0                   # a NaN
    x[0, 1, 0:4] = bf16_rne_bits([6.0, -6.5, 3.0, 2.0 ** -130])
    q, s = fp4.quantize_mx(x)
    assert list(s[0, 0]) == [255, 127] and list(s[0, 1]) == [127, 255]
    assert list(fp4.unpack(q)[0, 1, :4]) == [7, 15, 5, 0]
    q, s, gs = fp4.quantize_nv(x)
    assert gs[0] == np.float32(6.5) / np.float32(2688)
    assert list(s[0, 0]) == [0x7F, 0, 0, 0] and s[0, 1, 0] == 0x7E and s[0, 1, 2] == 0x7F
    tiny = bf16_rne_bits(np.full((1, 1, 32), 2.0 ** -133))
    q, s = fp4.quantize_mx(tiny)
    assert s[0, 0, 0] == 0 and np.all(fp4.unpack(q) == 0)
    assert np.isnan(fp4.decode_f64(np.zeros((1, 16), np.uint8), np.array([[255]], np.uint8), False)).all()


def test_grouped_gradients_are_adjoint():
    rng = np.random.default_rng(6)
    off = [0, 3, 3, 10]
    A, W, dC = rng.standard_normal((10, 5)), rng.standard_normal((3, 7, 5)), rng.standard_normal((10, 7))
    T = lambda v: torch.tensor(v, requires_grad=True)
    At, Wt = T(A), T(W)
    out = torch.cat([At[off[e]:off[e + 1]] @ Wt[e].t() for e in range(3)])
    (out * torch.tensor(dC)).sum().backward()
    assert np.allclose(grouped.forward_f64(A, W, off), out.detach().numpy())
    assert np.allclose(grouped.dgrad_f64(dC, W, off), At.grad.numpy())
    assert np.allclose(grouped.wgrad_f64(dC, A, off), Wt.grad.numpy())
    assert np.all(grouped.wgrad_f64(dC, A, off)[1] == 0)
    assert np.isnan(grouped.forward_f64(np.ones((12, 5)), W, off)[10:]).all()
    d, e = rng.standard_normal(A.shape), 1e-6      # differences along one direction
    f = lambda a: float(np.sum(grouped.forward_f64(a, W, off) * dC))
    assert abs((f(A + e * d) - f(A - e * d)) / (2 * e) - np.sum(d * grouped.dgrad_f64(dC, W, off))) < 1e-7


def test_clip_closed_forms():
    t = [np.array([3.0, 0.0]), np.array([[4.0]])]
    n, c, out = grouped.clip_f64(t, 1.0, 0.0)
    assert n == 5.0 and c == 0.2 and out[1][0, 0] == 0.8
    assert grouped.clip_f64(t, 5.0, 0.0)[1] == 1.0 and grouped.clip_f64(t, 50.0, 1e-6)[1] == 1.0
    assert grouped.clip_f64([], 1.0, 1e-6)[:2] == (0.0, 1.0)
    params = [torch.nn.Parameter(torch.zeros(2)), torch.nn.Parameter(torch.zeros(1, 1))]
    for p, g in zip(params, t):
        p.grad = torch.tensor(g, dtype=torch.float32).clone()
    assert float(torch.nn.utils.clip_grad_norm_(params, 1.0)) == 5.0
    for p, g in zip(params, grouped.clip_f64(t, 1.0, 1e-6)[2]):
        assert np.allclose(p.grad.numpy(), g, rtol=1e-6)
