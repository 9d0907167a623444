"""SwiGLU with its 8-bit input copy, and the gradient from that copy, on the
GPU: the copy bit for bit, h and the gradients within an fp32 evaluation's
slack of the fp64 definition plus half a bf16 unit.  The slack is that of
silu(g) u: 2^-20 relative (an exponential and a reciprocal of a few units
each, up to six roundings) on the magnitudes added, and for g below -87,
where e^-g leaves fp32, the value's own bound 2^-118 |u| (1 + |g|)."""

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, checkpoint_ref, swiglu_backward_f64
from oracle.swiglu import swiglu_f64
from oracle.swiglu8 import decode_f64

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _half_ulp(v):
    _, p = np.frexp(np.abs(v))
    return np.ldexp(0.5, np.maximum(p - 8, -133))


def _input(R, I, seed):
    rng = np.random.default_rng(seed)
    C = rng.standard_normal((R, 2 * I)).astype(np.float32)
    C[:, :I] *= 4
    if R > 4:
        C[0, :128] = 0
        C[1, :I] = np.linspace(-130, 130, I)
        C[2] *= np.float32(2.0 ** -60)
        C[3, :128] = 2.0 ** -101                         # below what the copy keeps
        C[3, 128:256] = 2.0 ** -100
        C[4, I:] *= np.float32(2.0 ** 100)
    return torch.from_numpy(C).to(torch.bfloat16)


CASES = [(1, 128), (2, 256), (7, 384), (33, 1792), (130, 2048), (3, 8320)]


@pytest.mark.parametrize("R,I", CASES)
def test_forward_and_copy(gpu_lib, R, I):
    C = _input(R, I, R + I)
    h, codes, scales = gpu_lib.swiglu(C.cuda(), checkpoint=True)
    rc, rs = checkpoint_ref(_bits(C))
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    plain = gpu_lib.swiglu(C.cuda())
    assert torch.equal(plain, h)                         # the copy does not change h
    v = bf16_bits_to_f64(_bits(C))
    ref = swiglu_f64(v[:, :I], v[:, I:])
    slack = np.abs(ref) * 2.0 ** -20 + np.abs(v[:, I:]) * 2.0 ** -118
    err = np.abs(h.double().cpu().numpy() - ref)
    assert (err <= slack + _half_ulp(np.abs(ref) + slack)).all()


@pytest.mark.parametrize("R,I", CASES)
def test_backward(gpu_lib, R, I):
    C = _input(R, I, R + I + 1)
    rng = np.random.default_rng(R)
    dh = torch.from_numpy(rng.standard_normal((R, I), dtype=np.float32)).to(torch.bfloat16)
    codes, scales = checkpoint_ref(_bits(C))
    args = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), dh.cuda())
    h = torch.empty((R, I), dtype=torch.bfloat16, device="cuda")
    dC, h2 = gpu_lib.swiglu_backward(*args, h=h)
    assert h2 is h and torch.equal(gpu_lib.swiglu_backward(*args), dC)
    ref, rh = swiglu_backward_f64(codes, scales, dh.double().numpy())
    v = decode_f64(codes, scales)
    g, u, d = v[:, :I], v[:, I:], np.abs(dh.double().numpy())
    sg = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
    sl = np.concatenate([d * np.abs(u) * (sg * (1 + np.abs(g) * (1 - sg)) * 2.0 ** -20 + (1 + np.abs(g)) * 2.0 ** -118),
                         d * (np.abs(g) * sg * 2.0 ** -20 + (1 + np.abs(g)) * 2.0 ** -118)], axis=1)
    err = np.abs(dC.double().cpu().numpy() - ref)
    bound = sl + _half_ulp(np.abs(ref) + sl)
    print(f"R={R} I={I}: largest error / bound {(err / bound).max():.3f}", flush=True)
    assert (err <= bound).all()
    sl = np.abs(rh) * 2.0 ** -20 + np.abs(u) * (1 + np.abs(g)) * 2.0 ** -118
    assert (np.abs(h.double().cpu().numpy() - rh) <= sl + _half_ulp(np.abs(rh) + sl)).all()


def test_gradient_against_differences_of_the_definition(gpu_lib):
    C = _input(3, 128, 9)
    codes, scales = checkpoint_ref(_bits(C))
    dh = torch.ones((3, 128), dtype=torch.bfloat16)
    dC = gpu_lib.swiglu_backward(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
                                 dh.cuda()).double().cpu().numpy()
    v = decode_f64(codes, scales)
    f = lambda a: (a[:, :128] / (1 + np.exp(-a[:, :128])) * a[:, 128:])  # noqa: E731
    for part in (0, 1):
        e = np.zeros(256)
        e[128 * part:128 * (part + 1)] = 1e-5
        num = (f(v + e) - f(v - e)) / 2e-5
        got = dC[:, 128 * part:128 * (part + 1)]
        assert (np.abs(got - num) <= np.abs(num) * 2.0 ** -8 + 1e-6).all()


def test_nan_and_infinity_reach_the_copy(gpu_lib):
    C = _input(2, 256, 10)
    C[0, 5], C[1, 300] = float("nan"), float("inf")
    h, codes, scales = gpu_lib.swiglu(C.cuda(), checkpoint=True)
    assert torch.isnan(h[0, 5]) and int((~torch.isfinite(h)).sum()) == 2
    v = codes.view(torch.float8_e4m3fn).float().view(2, 4, 128) * scales.view(2, 4, 1)
    assert torch.isnan(v[0, 0, 5]) and int(torch.isnan(v[0]).sum()) == 1
    assert torch.isnan(v[1, 2]).all() and torch.isfinite(v[1, [0, 1, 3]]).all()
    dC = gpu_lib.swiglu_backward(codes, scales, torch.ones_like(h))
    bad = ~torch.isfinite(dC)
    assert bad[0, 5] and bad[0, 261] and int(bad[0].sum()) == 2
    assert bad[1, 44:172].sum() >= 128 - 44 and not bad[1, 128:256].any()


def test_offsets_past_32_bits(gpu_lib):
    """The last of 600000 rows of 2 x 2048: element offsets past 2^31, byte offsets past 2^32."""
    R, I = 600000, 2048
    C = torch.zeros((R, 2 * I), dtype=torch.bfloat16, device="cuda")
    last = _input(1, I, 11)
    C[R - 1:] = last.cuda()
    h, codes, scales = gpu_lib.swiglu(C, checkpoint=True)
    rc, rs = checkpoint_ref(_bits(last))
    assert np.array_equal(codes[R - 1:].cpu().numpy(), rc) and np.array_equal(scales[R - 1:].cpu().numpy(), rs)
    del C
    dC = gpu_lib.swiglu_backward(codes, scales, h)
    small = gpu_lib.swiglu_backward(codes[R - 1:].contiguous(), scales[R - 1:].contiguous(), h[R - 1:].contiguous())
    assert torch.equal(dC[R - 1:], small) and not dC[:8].any()


def test_empty_stream_and_refusals(gpu_lib):
    z = torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda")
    h, c, s = gpu_lib.swiglu(z, checkpoint=True)
    assert h.shape == (0, 128) and c.shape == (0, 256) and s.shape == (0, 2)
    assert gpu_lib.swiglu_backward(c, s, h).shape == (0, 256)
    C = _input(5, 128, 12).cuda()
    want = gpu_lib.swiglu(C)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = gpu_lib.swiglu(C)
    side.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(gpu_lib.W4A8Error):
        gpu_lib.swiglu(torch.zeros((2, 200), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.swiglu(C, codes=torch.zeros((5, 256), dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        gpu_lib.swiglu(C.float())
    with pytest.raises(ValueError):
        gpu_lib.swiglu_backward(torch.zeros((5, 128), dtype=torch.uint8, device="cuda"),
                                torch.zeros((5, 2), device="cuda"), want)
