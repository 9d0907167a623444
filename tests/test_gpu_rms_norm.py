"""The norm with residual, its 8-bit output and its gradient on the GPU against
oracle/norm.py.

Bounds.  h: bit for bit.  y: the row's factor is an fp32 reciprocal root of a
64-bit sum with one Newton step (2^-23) in two factors, then three products
(2^-24 each): under 2^-21 of |y| before its rounding to bf16 (2^-8, and half a
subnormal step 2^-134).  Codes: admissible for a y off by 2^-21.  dx: m = mean(g
xh) has 64-bit sums of g rounded once (2^-24 of each term) and one rounding;
each element then four roundings beside its factor's: under 2^-20 of the
magnitudes n (|g| + |xh| mean|g xh|) + |dsum|, then bf16.  dw: an fp32 sum of at
most ceil(T / 1024) products per part, xh off by 2^-21, parts in 64 bits:
(ceil(T / 1024) + 10) 2^-24 of the magnitudes' sum."""

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, bf16_rne_bits, norm

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 8), (2, 7), (3, 64), (5, 100), (4, 128), (64, 6144), (37, 1001), (1025, 512), (9, 8192),
          (2, 8200), (3, 16384), (2, 16392), (2, 32768), (2, 32776), (3, 40001), (2, 65536), (2100, 136)]


def _dev(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _rows(T, K, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return bf16_rne_bits(rng.standard_normal((T, K)) * scale * (0.25 + rng.random((T, 1))))


def _weight(K, seed, kind):
    w = np.random.default_rng(seed).standard_normal(K)
    if kind == "none":
        return None, None
    if kind == "f32":
        w = w.astype(np.float32)
        return torch.from_numpy(w).cuda(), w.astype(np.float64)
    b = bf16_rne_bits(w)
    return _dev(b), bf16_bits_to_f64(b)


def _near_bf16(got, want, mag=None, rel=2.0 ** -21):
    bound = np.abs(want) * 2.0 ** -8 + 2.0 ** -134 + (np.abs(want) if mag is None else mag) * rel * (1 + 2.0 ** -8)
    g = bf16_bits_to_f64(_bits(got))
    assert g.shape == want.shape
    worst = np.max(np.abs(g - want) / bound) if g.size else 0.0
    assert worst <= 1.0, worst


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("kind,residual", [("bf16", True), ("f32", False), ("none", True)])
def test_norm(gpu_lib, T, K, kind, residual):
    x, r = _rows(T, K, T + K), _rows(T, K, T + K + 1, 3.0)
    w, wf = _weight(K, K, kind)
    h = norm.sum_bits(x, r if residual else None)
    got = gpu_lib.rms_norm(_dev(x), w, 1e-5, residual=_dev(r) if residual else None)
    y = got[0] if residual else got
    if residual:
        assert np.array_equal(_bits(got[1]), h)
    _near_bf16(y, norm.rms_norm_f64(h, wf, 1e-5))


@pytest.mark.parametrize("T,K", [(1, 128), (3, 256), (64, 6144), (64, 2048), (37, 1152), (1032, 384), (9, 8192),
                                 (2, 33280), (8, 16512)])
@pytest.mark.parametrize("layout", [0, 1])
def test_norm_in_8_bits(gpu_lib, T, K, layout):
    x, r = _rows(T, K, T * K), _rows(T, K, T * K + 1)
    x[0, :128] = 0
    r[0, :128] = 0                                      # a group of zeros: scale 1
    w, wf = _weight(K, K, "bf16")
    h = norm.sum_bits(x, r)
    out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    A, SA, H = gpu_lib.rms_norm_quant(_dev(x), w, layout, 1e-6, residual=_dev(r), out=out)
    assert np.array_equal(_bits(H), h)
    y = norm.rms_norm_f64(h, wf, 1e-6)
    s = SA.cpu().numpy()
    assert s.shape == ((T, K // 128) if layout == 0 else (K // 128, T))
    assert norm.check_codes(A.cpu().numpy(), s if layout == 0 else s.T, y, 2.0 ** -21) == 0
    assert s.reshape(-1)[0] == 1.0 and np.all(A.cpu().numpy()[0, :128] & 0x7F == 0)
    _near_bf16(out, y)


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("kind,dsum", [("bf16", True), ("f32", False), ("none", False)])
def test_norm_backward(gpu_lib, T, K, kind, dsum):
    h, dy, r = _rows(T, K, T + K), _rows(T, K, T + K + 1, 0.1), _rows(T, K, T + K + 2, 0.1)
    w, wf = _weight(K, K, kind)
    dx, dw, mag, wmag = norm.rms_norm_backward_f64(h, wf, dy, 1e-5, r if dsum else None)
    gx, gw = gpu_lib.rms_norm_backward(_dev(h), w, _dev(dy), 1e-5, dh=_dev(r) if dsum else None)
    _near_bf16(gx, dx, mag, 2.0 ** -20)
    bound = (-(-T // 1024) + 10) * 2.0 ** -24 * wmag + 2.0 ** -149
    assert np.max(np.abs(gw.cpu().numpy() - dw) / bound) <= 1.0
    again = gpu_lib.rms_norm_backward(_dev(h), w, _dev(dy), 1e-5, dh=_dev(r) if dsum else None)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** 64, 2.0 ** -60, 2.0 ** -100])
def test_range(gpu_lib, scale):
    """Rows whose squares are past fp32's range, with eps = 0: y does not change with a power of two."""
    x = _rows(4, 512, 5)
    xs = bf16_rne_bits(bf16_bits_to_f64(x) * scale)
    a, b = gpu_lib.rms_norm(_dev(xs), None, 0.0), gpu_lib.rms_norm(_dev(x), None, 0.0)
    assert torch.equal(a, b)
    dy = _rows(4, 512, 6)
    dx, dw, mag, wmag = norm.rms_norm_backward_f64(xs, None, dy, 0.0)
    gx, gw = gpu_lib.rms_norm_backward(_dev(xs), None, _dev(dy), 0.0)
    _near_bf16(gx, dx, mag, 2.0 ** -20)
    assert np.all(np.abs(gw.cpu().numpy() - dw) <= 11 * 2.0 ** -24 * wmag)


def test_special_rows(gpu_lib):
    x = _rows(6, 256, 7)
    x[0] = 0
    x[1, 5] = 0x7F80
    x[2, 6] = 0x7FC0
    x[3] = 0x7F7F                                       # all at bf16's largest value
    y = gpu_lib.rms_norm(_dev(x), None, 0.0).float().cpu()
    assert torch.isnan(y[0]).all()                      # 0 / 0
    assert torch.isnan(y[1, 5]) and (y[1, :5] == 0).all() and torch.isnan(y[2]).all()
    assert (y[3] == 1.0).all()
    want = norm.rms_norm_f64(x[4:], None, 0.0)
    assert np.allclose(y[4:].numpy(), want, rtol=2.0 ** -7)
    assert (gpu_lib.rms_norm(_dev(x[:1]), None, 1e-6) == 0).all()
    A, SA = gpu_lib.rms_norm_quant(_dev(x), None, 0, 0.0)
    v = A.view(torch.float8_e4m3fn).float().view(6, 2, 128) * SA[:, :, None]
    assert torch.isnan(v[0]).all() and torch.isnan(v[2]).all() and torch.isnan(v[1].reshape(-1)[5])
    assert torch.isfinite(v[3:]).all()


def test_in_place_unaligned_and_side_stream(gpu_lib):
    T, K = 33, 520
    x, r = _rows(T, K, 8), _rows(T, K, 9)
    y0, h0 = gpu_lib.rms_norm(_dev(x), None, 1e-6, residual=_dev(r))
    buf = torch.zeros(2 * T * K + 8, dtype=torch.bfloat16, device="cuda")
    xs, rs = buf[1:1 + T * K].view(T, K), buf[T * K + 3:2 * T * K + 3].view(T, K)
    xs.copy_(_dev(x))
    rs.copy_(_dev(r))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, h = gpu_lib.rms_norm(xs, None, 1e-6, residual=rs, out=xs, sum_out=rs)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y0) and torch.equal(h, h0) and y.data_ptr() == xs.data_ptr()
    assert float(buf[0]) == 0 and (buf[1 + T * K:T * K + 3] == 0).all() and (buf[2 * T * K + 3:] == 0).all()
    dy = _dev(_rows(T, K, 10))
    dx0, dw0 = gpu_lib.rms_norm_backward(h0, None, dy)
    dx, dw = gpu_lib.rms_norm_backward(h0, None, dy, dx=dy)
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0) and dx.data_ptr() == dy.data_ptr()
    big = _rows(2, 40000, 11)                           # the two-pass kernel in place
    y0, h0 = gpu_lib.rms_norm(_dev(big), None, 1e-6, residual=_dev(big))
    a, b = _dev(big), _dev(big)
    y, h = gpu_lib.rms_norm(a, None, 1e-6, residual=b, out=b, sum_out=a)
    assert torch.equal(y, y0) and torch.equal(h, h0)


def test_no_rows_and_refusals(gpu_lib):
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    assert gpu_lib.rms_norm(e).shape == (0, 256)
    dx, dw = gpu_lib.rms_norm_backward(e, None, e, dweight=torch.full((256,), 7.0, device="cuda"))
    assert dx.shape == (0, 256) and (dw == 0).all()
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        gpu_lib.rms_norm(x, sum_out=x)
    with pytest.raises(ValueError):
        gpu_lib.rms_norm(x.t())
    with pytest.raises(TypeError):
        gpu_lib.rms_norm(x, torch.ones(256, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.rms_norm(x, torch.ones(255, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.rms_norm_quant(x[:, :64].contiguous(), None, 0)
    with pytest.raises(gpu_lib.W4A8Error):
        gpu_lib.rms_norm(x, None, -1.0)
    with pytest.raises(gpu_lib.W4A8Error):
        gpu_lib.rms_norm_backward(x, None, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_offsets_past_32_bits(gpu_lib):
    T, K = 270000, 8192                                 # 2.2e9 elements
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[-1] = 2.0
    x[-2, 0] = 3.0
    y = gpu_lib.rms_norm(x, None, 0.25, out=x)
    assert y.data_ptr() == x.data_ptr() and (y[:2] == 0).all()
    assert torch.allclose(y[-1].float(), torch.full((K,), 2.0 / 4.25 ** 0.5, device="cuda"), rtol=2.0 ** -8)
    assert float(y[-3].abs().max()) == 0.0 and (y[-2, 1:] == 0).all() and float(y[-2, 0]) > 1.0
