"""The norm over many tensors and their scaling on the GPU against
oracle/grouped.py clip_f64.

Bounds: the norm is a 64-bit sum rounded to fp32 (2^-24; 2^-23 asked); an
output is c x with c rounded (2^-24) and the product rounded (2^-24), then its
type (bf16 2^-8 and half a subnormal step)."""

import math

import numpy as np
import pytest
import torch

from oracle import grouped

pytestmark = pytest.mark.gpu


def _tensors(sizes, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale).to(torch.float32 if i % 2 else torch.bfloat16).cuda()
            for i, s in enumerate(sizes)]


def _np(t):
    return t.double().cpu().numpy()


def _check(lib, ts, max_norm, eps=1e-6):
    norm, c, want = grouped.clip_f64([_np(t) for t in ts], max_norm, eps)
    outs = [torch.full_like(t, 9.0) for t in ts]
    before = [t.clone() for t in ts]
    n1 = lib.grad_norm(ts)
    n2 = lib.clip_grads(ts, max_norm, eps, out=outs)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    n3 = lib.clip_grads(ts, max_norm, eps)
    assert n1.shape == (1,) and torch.equal(n1, n2) and torch.equal(n1, n3)
    assert abs(float(n1) - norm) <= norm * 2.0 ** -23
    for t, o, w, b in zip(ts, outs, want, before):
        assert torch.equal(t, o)
        bound = np.abs(w) * (2.0 ** -22 + (2.0 ** -8 if t.dtype == torch.bfloat16 else 0)) + 2.0 ** -134
        assert np.all(np.abs(_np(t) - w) <= bound)
        if c == 1.0:
            assert torch.equal(t, b)


SIZES = [[(1,)], [(3,), (5, 7), (1,)], [(8192,), (8193,), (8191,), (1, 2, 3)], [(100000,), (0,), (33, 1001)],
         [(n,) for n in range(1, 96)], [(17 * n,) for n in range(1, 97)], [(n,) for n in range(1, 98)],
         [(5,)] * 300, [(3000000,), (2, 512, 768)], [(0,), (0, 4)], []]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
def test_clip(gpu_lib, sizes, max_norm):
    _check(gpu_lib, _tensors(sizes, len(sizes)), max_norm)


def test_range(gpu_lib):
    for scale in (1e30, 1e-30):                          # squares past fp32 on both sides
        _check(gpu_lib, _tensors([(1000,), (77,), (40, 3)], 1, scale), scale)
    t = [torch.full((1 << 16,), 3e38, device="cuda")]    # the norm itself past fp32
    assert math.isinf(float(gpu_lib.clip_grads(t, 1.0)))
    assert torch.allclose(t[0], torch.full_like(t[0], 1.0 / 256), rtol=2.0 ** -22)


def test_non_finite(gpu_lib):
    t = _tensors([(100,), (50,)], 2)
    t[0][3] = float("inf")
    assert math.isinf(float(gpu_lib.clip_grads(t, 1.0)))
    assert torch.isnan(t[0][3]) and (t[1] == 0).all() and (t[0][:3] == 0).all()
    t = _tensors([(100,), (50,)], 3)
    t[1][7] = float("nan")
    assert math.isnan(float(gpu_lib.clip_grads(t, 1.0)))
    assert all(torch.isnan(v).all() for v in t)


def test_unaligned_views(gpu_lib):
    b16 = torch.randn(5000, device="cuda").bfloat16()
    b32 = torch.randn(5000, device="cuda")
    views = [b16[1:2000], b16[2001:2009], b32[3:4000], b32[4001:]]
    keep = b16.clone(), b32.clone()
    _check(gpu_lib, views, 0.25)
    for b, k in zip((b16, b32), keep):
        assert torch.equal(b[:1], k[:1])
    assert torch.equal(b16[2000], keep[0][2000]) and torch.equal(b32[4000], keep[1][4000])


def test_repeats_and_streams(gpu_lib):
    ts = _tensors([(100001,), (64, 999)], 4)
    want = gpu_lib.grad_norm(ts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [gpu_lib.grad_norm(ts) for _ in range(5)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_refusals(gpu_lib):
    t = torch.ones(64, device="cuda")
    for call in (lambda: gpu_lib.clip_grads([t, t], 1.0), lambda: gpu_lib.clip_grads([t, t[32:]], 1.0),
                 lambda: gpu_lib.clip_grads([t[:32], t[32:]], 1.0, out=[t[32:], t[:32]]),
                 lambda: gpu_lib.clip_grads([t], -1.0), lambda: gpu_lib.clip_grads([t], float("nan")),
                 lambda: gpu_lib.clip_grads([t], 1.0, eps=-1.0),
                 lambda: gpu_lib.grad_norm([t], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gpu_lib.W4A8Error):
            call()
    for call in (lambda: gpu_lib.clip_grads([t], 1.0, out=[]), lambda: gpu_lib.clip_grads([t.cpu()], 1.0),
                 lambda: gpu_lib.clip_grads([t.view(8, 8).t()], 1.0),
                 lambda: gpu_lib.clip_grads([t], 1.0, out=[t[:63]])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gpu_lib.clip_grads([t.half()], 1.0), lambda: gpu_lib.clip_grads([t], 1.0, out=[t.bfloat16()])):
        with pytest.raises(TypeError):
            call()
    assert (t == 1).all()
    assert float(gpu_lib.grad_norm([t, t])) == np.float32(math.sqrt(128))      # a sum may have a tensor twice
