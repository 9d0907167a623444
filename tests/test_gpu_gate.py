"""Router gate on the GPU (w4a8_topk_gate, w4a8_topk_gate_backward) against
the fp64 oracle: ids equal, weights and gradients within their fp32 bounds.

Bounds, with D the row's spread of finite logits: e^(l - m) carries the
rounding of l - m (at most D 2^-24 absolute in the exponent) and a few units
of exp; a sum of up to 16384 terms in a tree of 16 per lane and 10 levels, a
division and the scale add less than 40 units; the sigmoid and its ratio
form stay within the same.  So a weight is within (D + 64) 2^-23 relative,
and a gradient within (D + 128) 2^-22 of the magnitudes that it subtracts."""

import numpy as np
import pytest
import torch

from oracle import topk_gate_backward_f64, topk_gate_f64

pytestmark = pytest.mark.gpu

MODES = [(0, False), (0, True), (1, False), (1, True)]
SHAPES = [(1, 1, 1), (1, 2, 2), (5, 4, 1), (64, 32, 8), (33, 64, 64), (7, 65, 5), (9, 200, 12), (6, 333, 8),
          (5, 1000, 8), (3, 1024, 64), (4, 1025, 8), (3, 2048, 8), (2, 6144, 64), (2, 6143, 7), (1, 16384, 33)]


def _logits(T, E, seed, bf16):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    l[rng.random((T, E)) < 0.15] = -np.inf
    if T > 2:
        l[1] = -np.inf                                        # a token with no expert
        l[2] = np.round(l[2])                                 # many ties
        l[0] = np.where(rng.random(E) < 0.5, np.finfo(np.float32).min if not bf16 else -3.3895314e38, l[0])
    if T > 4:
        l[3, min(3, E - 1):] = -np.inf                        # fewer left than top_k
        l[4] *= 25                                            # logits past both ends of the exponential
        l[4, ::3] = -150.0                                    # whose sigmoid is below fp32's range
    t = torch.from_numpy(l).to(torch.bfloat16 if bf16 else torch.float32)
    return t, t.double().numpy()


def _spread(l):
    f = np.where(np.isfinite(l) & (np.abs(l) < 1e30), l, np.nan)
    with np.errstate(all="ignore"):
        d = np.nan_to_num(np.nanmax(f, 1, initial=-1e30) - np.nanmin(f, 1, initial=1e30), neginf=0.0)
    return np.clip(d, 0, 300)[:, None]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gate_forward(gpu_lib, T, E, k, bf16):
    t, l = _logits(T, E, T * 1000 + E, bf16)
    for score, renorm in MODES:
        ids, w = gpu_lib.topk_gate(t.cuda(), k, score, renorm, 2.5)
        rids, rw = topk_gate_f64(l, k, score, renorm, 2.5)
        assert np.array_equal(ids.cpu().numpy(), rids)
        got = w.cpu().numpy().astype(np.float64)
        err = np.abs(got - rw)
        bound = rw * (_spread(l) + 64) * 2.0 ** -23 + 2.5 * 2.0 ** -125
        print(f"T={T} E={E} k={k} bf16={bf16} score={score} renorm={renorm}: largest error / bound "
              f"{(err / bound).max():.2f}", flush=True)
        assert (err <= bound).all()
        assert (got[rids < 0] == 0).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gate_backward(gpu_lib, T, E, k, bf16):
    t, l = _logits(T, E, T * 1000 + E + 1, bf16)
    rng = np.random.default_rng(E)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for score, renorm in MODES:
        ids, rw = topk_gate_f64(l, k, score, renorm)
        ref = topk_gate_backward_f64(l, ids, dw, score, renorm, 0.5)
        d = gpu_lib.topk_gate_backward(t.cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), score,
                                       renorm, 0.5)
        assert d.dtype == t.dtype
        got = d.double().cpu().numpy()
        # what an element subtracts: its own weight times (its g + the weighted sum)
        g = 0.5 * np.abs(dw) * (ids >= 0)
        dot = (g * rw).sum(1, keepdims=True)
        p = np.zeros_like(l)
        if score == 0 and not renorm:
            with np.errstate(invalid="ignore"):
                p = np.nan_to_num(np.exp(l - l.max(1, keepdims=True)))
                p = np.nan_to_num(p / p.sum(1, keepdims=True))
        G = np.zeros_like(l)
        for r in range(T):
            ok = ids[r] >= 0
            G[r, ids[r][ok]] = g[r, ok] * rw[r, ok]
            if renorm or score == 1:
                p[r, ids[r][ok]] = rw[r, ok]
        bound = (G + p * dot) * (_spread(l) + 128) * 2.0 ** -22 + 2.0 ** -120
        if bf16:
            bound = bound + np.abs(ref) * 2.0 ** -8
        err = np.abs(got - ref)
        print(f"T={T} E={E} k={k} bf16={bf16} score={score} renorm={renorm}: largest error / bound "
              f"{(err / bound).max():.2f}", flush=True)
        assert (err <= bound).all()


def test_gate_gradient_against_differences(gpu_lib):
    """Central differences of the device's own forward pass: h = 2^-6 costs
    h^2 / 6 times a third derivative below 2 in size, the fp32 weights
    2^-22 / h; together below 2e-4."""
    rng = np.random.default_rng(3)
    l = rng.standard_normal((4, 10)).astype(np.float32)
    dw = rng.standard_normal((4, 3)).astype(np.float32)
    h = 2.0 ** -6
    for score, renorm in MODES:
        ids, _ = gpu_lib.topk_gate(torch.from_numpy(l).cuda(), 10, score, False)
        ids3 = ids[:, :3].contiguous()
        d = gpu_lib.topk_gate_backward(torch.from_numpy(l).cuda(), ids3, torch.from_numpy(dw).cuda(), score,
                                       renorm).cpu().numpy()

        def weighted(a):   # the selection held fixed: take the weights at ids3 from a full ranking
            i, w = gpu_lib.topk_gate(torch.from_numpy(a.astype(np.float32)).cuda(), 10, score, False)
            full = torch.zeros((4, 10), dtype=torch.float64, device="cuda").scatter_(1, i.long(), w.double())
            v = full.gather(1, ids3.long())
            if renorm:
                v = v / v.sum(1, keepdim=True)
            return (v.cpu().numpy() * dw).sum(1)
        for e in range(10):
            a, b = l.copy(), l.copy()
            a[:, e] += h
            b[:, e] -= h
            num = (weighted(a) - weighted(b)) / ((a - b)[:, e].astype(np.float64))
            assert np.abs(num - d[:, e]).max() < 2e-4


def test_gate_nan_and_infinity(gpu_lib):
    inf, nan = float("inf"), float("nan")
    l = torch.tensor([[0.0, nan, 1.0, -inf], [0.0, inf, 1.0, -inf], [-0.0, 0.0, -inf, -inf]])
    ids, w = gpu_lib.topk_gate(l.cuda(), 3, 0, True)
    assert ids.tolist() == [[1, 2, 0], [1, 2, 0], [0, 1, -1]]
    assert torch.isnan(w[:2]).all() and w[2].tolist() == [0.5, 0.5, 0.0]
    ids, w = gpu_lib.topk_gate(l.cuda(), 3, 1, False)
    assert torch.isnan(w[0, 0]) and not torch.isnan(w[0, 1:]).any() and w[1, 0] == 1
    for score, renorm in MODES:
        i, a = gpu_lib.topk_gate(l.cuda(), 3, score, renorm)
        j, b = topk_gate_f64(l.double().numpy(), 3, score, renorm)
        assert np.array_equal(i.cpu().numpy(), j) and np.array_equal(np.isnan(a.cpu().numpy()), np.isnan(b))


def test_gate_backward_ignores_foreign_ids_and_their_gradients(gpu_lib):
    l = torch.randn((2, 70), generator=torch.Generator().manual_seed(1))
    ids = torch.tensor([[3, -1, 69], [70, 5, 1 << 30]], dtype=torch.int32)
    nan = float("nan")
    dw = torch.tensor([[1.0, nan, 2.0], [nan, 3.0, nan]])
    for score, renorm in MODES:
        d = gpu_lib.topk_gate_backward(l.cuda(), ids.cuda(), dw.cuda(), score, renorm).cpu().double().numpy()
        clean = np.where(ids.numpy() >= 70, -1, ids.numpy())
        ref = topk_gate_backward_f64(l.double().numpy(), clean, np.nan_to_num(dw.numpy()), score, renorm)
        assert np.allclose(d, ref, rtol=1e-5, atol=1e-7)


def test_gate_misaligned_rows_stream_and_repeat(gpu_lib):
    """Rows that start at any element, a side stream, and equal bits on every call."""
    flat = torch.randn(1 + 40 * 333, generator=torch.Generator().manual_seed(2)).cuda()
    for dt in (torch.float32, torch.bfloat16):
        l = flat.to(dt)[1:].view(40, 333)
        want = gpu_lib.topk_gate(l.clone(), 8)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = gpu_lib.topk_gate(l, 8)
            d1 = gpu_lib.topk_gate_backward(l, got[0], got[1], 0, False)
        torch.cuda.current_stream().wait_stream(side)
        d2 = gpu_lib.topk_gate_backward(l.clone(), want[0], want[1], 0, False)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(d1, d2)


def test_gate_empty_and_refusals(gpu_lib):
    e = torch.zeros((0, 8), device="cuda")
    ids, w = gpu_lib.topk_gate(e, 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert gpu_lib.topk_gate_backward(e, ids, w).shape == (0, 8)
    l = torch.zeros((4, 8), device="cuda")
    for bad in (lambda: gpu_lib.topk_gate(l, 9), lambda: gpu_lib.topk_gate(l, 0),
                lambda: gpu_lib.topk_gate(l, 2, score=7)):
        with pytest.raises(gpu_lib.W4A8Error):
            bad()
    with pytest.raises(TypeError):
        gpu_lib.topk_gate(l.half(), 2)
    with pytest.raises(ValueError):
        gpu_lib.topk_gate(l.t(), 2)                     # not contiguous
    with pytest.raises(ValueError):
        gpu_lib.topk_gate_backward(l, torch.zeros((3, 2), dtype=torch.int32, device="cuda"),
                                   torch.zeros((3, 2), device="cuda"))
