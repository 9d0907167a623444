"""Clipping where the factor max_norm / (norm + eps) is below fp32's normal
range, and at its border with 1, against oracle/grouped.py clip_f64.

Bounds: the factor is held to 24 bits (2^-24) and a product is rounded once
(2^-24), so 2^-22 of the value covers both and their product; the power of two
that follows is exact but for results below fp32's normal range (half a step of
2^-149, and the earlier rounding: one step asked); bf16 adds 2^-8 of the value
and one step of 2^-133."""

import numpy as np
import pytest
import torch

from oracle import grouped

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _tensors(scale, seed=0):
    """fp32 and bf16, whole 16-byte pieces and ends, a few elements many binades below the others."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate((70000, 4099, 13, 65536)):
        t = (torch.rand(n, generator=g, dtype=torch.float64) - 0.5) * scale
        t[::7] *= 2.0 ** -20
        out.append(t.to(torch.float32 if i % 2 else torch.bfloat16).cuda())
    return out


def _check(ts, got, want):
    for t, o, w in zip(ts, got, want):
        g, bf = _np(o), t.dtype == torch.bfloat16
        bound = np.abs(w) * (2.0 ** -22 + (2.0 ** -8 if bf else 0.0)) + (2.0 ** -133 if bf else 2.0 ** -149)
        worst = float(np.max(np.abs(g - w) / bound))
        assert worst <= 1.0, (t.dtype, worst)


@pytest.mark.parametrize("scale", [3e38, 1e36, 1e30])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-12, 1e-36, 2.0 ** -149])
def test_factors_below_the_normal_range(gpu_lib, scale, max_norm):
    ts = _tensors(scale)
    norm, c, want = grouped.clip_f64([_np(t) for t in ts], max_norm, 1e-6)
    out = [torch.full_like(t, 9.0) for t in ts]
    n = gpu_lib.clip_grads(ts, max_norm, out=out)
    _check(ts, out, want)
    m = gpu_lib.clip_grads(ts, max_norm)                # in place: the same
    assert torch.equal(n, m) and all(torch.equal(t, o) for t, o in zip(ts, out))
    many = [t for t in _tensors(scale) for t in t.chunk(40)]   # more tensors than a launch takes: other kernels
    _, _, want = grouped.clip_f64([_np(t) for t in many], max_norm, 1e-6)
    out = [torch.full_like(t, 9.0) for t in many]
    gpu_lib.clip_grads(many, max_norm, out=out)
    _check(many, out, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norms_next_to_max_norm(gpu_lib, dtype):
    """The factor is max_norm / (norm + eps): below 1 for a norm of max_norm itself, 1 without eps, and 1 for norms
    that are eps or more below; in place and with outputs of their own."""
    t0 = [torch.full((16,), v, dtype=dtype, device="cuda") for v in (0.5, -0.75, 1.5)]   # norm^2 = 49
    eps = 2.0 ** -10
    for max_norm, e, factor in ((7.0, eps, 7.0 / (7.0 + eps)), (7.0, 0.0, 1.0), (7.0 + eps, eps, 1.0),
                                (7.0 + 2 * eps, eps, 1.0), (6.5, 0.0, 6.5 / 7.0), (7.0, 1e-9, 1.0)):
        want = [(t.double() * factor) for t in t0]
        ts, out = [t.clone() for t in t0], [torch.full_like(t, 9.0) for t in t0]
        n = gpu_lib.clip_grads(ts, max_norm, e, out=out)
        assert float(n) == 7.0 and all(torch.equal(a, b) for a, b in zip(ts, t0))
        if factor == 1.0:
            assert all(torch.equal(a, b) for a, b in zip(out, t0))
        else:
            _check(ts, out, [_np(w) for w in want])
            if dtype is torch.float32:
                assert not any((a == b).any() for a, b in zip(out, t0))
        gpu_lib.clip_grads(ts, max_norm, e)
        assert all(torch.equal(a, b) for a, b in zip(ts, out))
