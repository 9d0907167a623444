"""The SwiGLU gradient over the whole range of gates that the 8-bit copy can
hold, against the fp64 definition.

Bound: the fp32 evaluation's 2^-20 relative on the magnitudes added, half a
bf16 unit, and what a sigmoid below fp32's range costs.  Below g = -88 the
device may take s up to e^-88 < 2^-126 for anything smaller, and s vanishes
below -104, so g s is within 104 * 2^-126 < 2^-119 of its value whatever |g|
(no factor |g|: the definition goes to zero there)."""

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, checkpoint_ref, swiglu_backward_f64
from oracle.swiglu import swiglu_f64
from oracle.swiglu8 import decode_f64

pytestmark = pytest.mark.gpu

I = 256


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _half_ulp(v):
    _, p = np.frexp(np.abs(v))
    return np.ldexp(0.5, np.maximum(p - 8, -133))


def _check(lib, C, dh):
    codes, scales = checkpoint_ref(_bits(C))
    h = torch.empty(dh.shape, dtype=torch.bfloat16, device="cuda")
    dC, h = lib.swiglu_backward(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), dh.cuda(), h=h)
    d = dh.double().numpy()
    ref, rh = swiglu_backward_f64(codes, scales, d)
    v = decode_f64(codes, scales)
    g, u, d = v[:, :I], np.abs(v[:, I:]), np.abs(d)
    e = np.exp(-np.abs(g))
    sg = np.where(g >= 0, 1 / (1 + e), e / (1 + e))
    one = np.where(g >= 0, e / (1 + e), 1 / (1 + e))         # 1 - sg
    tiny = 2.0 ** -118
    sl = np.concatenate([d * u * (sg * (1 + np.abs(g) * one) * 2.0 ** -20 + tiny),
                         d * (np.abs(g) * sg * 2.0 ** -20 + tiny)], axis=1)
    got, bound = dC.double().cpu().numpy(), sl + _half_ulp(np.abs(ref) + sl)
    err = np.abs(got - ref)
    print(f"dC: {int((~np.isfinite(got)).sum())} not finite, largest error / bound {np.nanmax(err / bound):.3g}", flush=True)
    assert (err <= bound).all()
    sl = np.abs(rh) * 2.0 ** -20 + u * tiny
    err, bound = np.abs(h.double().cpu().numpy() - rh), sl + _half_ulp(np.abs(rh) + sl)
    print(f"h: largest error / bound {np.nanmax(err / bound):.3g}", flush=True)
    assert (err <= bound).all()


@pytest.mark.parametrize("amax", [86.0, 89.0, 96.0, 105.0, 3e4, 3e7, 1e8, 2e8, 1e9, 1e12, 1e30, 3.3e38])
@pytest.mark.parametrize("sign", [-1, 1, 0])
def test_gates_of_any_size(gpu_lib, amax, sign):
    """Groups up to amax, one sign or both; u and dh below 1/2, so that no value overflows."""
    rng = np.random.default_rng(int(np.log2(amax)) * 3 + sign)
    C = np.empty((8, 2 * I))
    C[:, :I] = amax * rng.uniform(0, 1, (8, I)) * (sign if sign else rng.choice([-1, 1], (8, I)))
    C[:, 0] = C[:, 128] = amax * (sign or 1)
    C[:, I:] = rng.uniform(-0.5, 0.5, (8, I))
    C = torch.from_numpy(C.astype(np.float32)).to(torch.bfloat16)
    dh = torch.from_numpy(rng.uniform(-0.5, 0.5, (8, I)).astype(np.float32)).to(torch.bfloat16)
    _check(gpu_lib, C, dh)
    v = bf16_bits_to_f64(_bits(C))
    ref = swiglu_f64(v[:, :I], v[:, I:])
    got = gpu_lib.swiglu(C.cuda()).double().cpu().numpy()
    sl = np.abs(ref) * 2.0 ** -20 + np.abs(v[:, I:]) * 2.0 ** -118
    assert (np.abs(got - ref) <= sl + _half_ulp(np.abs(ref) + sl)).all()


def test_known_gates_of_the_rounding_correction(gpu_lib):
    """Gates where the rounding error of code * scale is itself 1.5 and 1:
    the gate's half of dC and h are 0 there."""
    for amax, code in ((65011712.0, -288.0), (30408704.0, -384.0)):
        scale = np.float32(amax) / np.float32(448.0)
        scales = torch.tensor([[float(scale), 1.0 / 448]] * 2)
        codes = torch.full((2, 256), code)
        codes[:, 128:] = 448.0
        codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        dh = torch.ones((2, 128), dtype=torch.bfloat16)
        h = torch.empty_like(dh).cuda()
        dC, h = gpu_lib.swiglu_backward(codes.cuda(), scales.cuda(), dh.cuda(), h=h)
        assert not dC.any() and not h.any()


def test_products_that_leave_fp32_in_between(gpu_lib):
    """dh u is past fp32's largest value, dh u s (1 + g (1 - s)) is not."""
    rng = np.random.default_rng(5)
    C = np.empty((6, 2 * I))
    C[:, :I] = rng.uniform(-80, -60, (6, I))
    C[:, I:] = rng.uniform(-1, 1, (6, I)) * 2.0 ** 100
    dh = rng.uniform(-1, 1, (6, I)) * 2.0 ** 70
    _check(gpu_lib, torch.from_numpy(C.astype(np.float32)).to(torch.bfloat16),
           torch.from_numpy(dh.astype(np.float32)).to(torch.bfloat16))
