"""A block whose experts are trained, run through the operators one after the
other as a training step does: norm with residual, gate, route prep, dispatch,
grouped products with bf16 weights around SwiGLU, combine, back through all of
them, clipping of the gradients, and the trained weights quantised to 4 bits and
multiplied by 4-bit rows.  Every step is compared with its oracle on the values
that the step before it gave, under that operator's own bound; the whole run is
captured in a graph and replayed bit for bit; and the gradient of the whole block
is compared along a direction with torch's autograd in fp64."""

import numpy as np
import pytest
import torch

from helpers import fp32_sum_eps
from oracle import bf16_bits_to_f64, fp4, grouped, norm

pytestmark = pytest.mark.gpu

T, H, I, E, K_TOP = 96, 256, 128, 8, 2
EPS = 1e-5


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def _f(t):
    return t.double().cpu().numpy()


@pytest.fixture
def block():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g)
    p = dict(w=1 + 0.1 * r(H), router=r(E, H) / H ** 0.5, w13=(r(E, 2 * I, H) / H ** 0.5).bfloat16(),
             w2=(r(E, H, I) / I ** 0.5).bfloat16(), x=r(T, H).bfloat16(), res=r(T, H).bfloat16(),
             dout=(0.1 * r(T, H)).bfloat16())
    return {k: v.cuda() for k, v in p.items()}


def _step(lib, p):
    """All intermediate values of a training step, by name."""
    v = {}
    v["y"], v["h"] = lib.rms_norm(p["x"], p["w"], EPS, residual=p["res"])
    v["logits"] = v["y"].float() @ p["router"].t()
    v["ids"], v["gw"] = lib.topk_gate(v["logits"], K_TOP)
    _, v["off"], v["rows"] = lib.route_prep(v["ids"], E)
    v["a"] = lib.dispatch(v["y"], v["rows"], K_TOP, T * K_TOP)
    v["c1"] = lib.grouped_gemm_bf16(v["a"], p["w13"], v["off"])
    v["h1"], v["codes"], v["scales"] = lib.swiglu(v["c1"], checkpoint=True)
    v["c2"] = lib.grouped_gemm_bf16(v["h1"], p["w2"], v["off"])
    v["out"] = lib.combine(v["c2"], v["rows"], v["gw"], K_TOP)
    v["dc2"], v["dgw"] = lib.combine_backward(v["c2"], p["dout"], v["rows"], v["gw"], K_TOP)
    v["dh1"] = lib.grouped_gemm_dgrad(v["dc2"], p["w2"], v["off"])
    v["dc1"], v["h1b"] = lib.swiglu_backward(v["codes"], v["scales"], v["dh1"], h=torch.empty_like(v["h1"]))
    v["dw2"] = lib.grouped_gemm_wgrad(v["dc2"], v["h1b"], v["off"])
    v["da"] = lib.grouped_gemm_dgrad(v["dc1"], p["w13"], v["off"])
    v["dw13"] = lib.grouped_gemm_wgrad(v["dc1"], v["a"], v["off"])
    v["dlogits"] = lib.topk_gate_backward(v["logits"], v["ids"], v["dgw"])
    v["dy"] = (lib.dispatch_backward(v["da"], v["rows"], K_TOP).float() + v["dlogits"] @ p["router"]).bfloat16()
    v["drouter"] = v["dlogits"].t() @ v["y"].float()
    v["dx"], v["dw"] = lib.rms_norm_backward(v["h"], p["w"], v["dy"], EPS, dh=p["dout"])
    v["clipped"] = [torch.empty_like(v[n]) for n in ("dw13", "dw2", "drouter", "dw")]
    v["norm"] = lib.clip_grads([v[n] for n in ("dw13", "dw2", "drouter", "dw")], 0.5, out=v["clipped"])
    v["b13"], v["sb13"], _ = lib.quantize_fp4(p["w13"], lib.WSCALE_MX)
    v["a4"], v["sa4"] = lib.quantize_gather_fp4(v["y"], v["rows"], K_TOP, T * K_TOP)
    v["c4"] = lib.grouped_gemm_a4(v["a4"], v["sa4"], v["b13"], v["sb13"], v["off"])
    return v


def _product(got, want, mag, Z, half):
    err = (Z + 8) * 2.0 ** -23 * mag
    assert np.all(np.abs(_f(got) - want) <= err + half * (np.abs(want) + err) + 2.0 ** -134)


def test_every_step_against_its_oracle(gpu_lib, block):
    v = _step(gpu_lib, block)
    w = _f(block["w"])
    h = norm.sum_bits(_bits(block["x"]), _bits(block["res"]))
    assert np.array_equal(_bits(v["h"]), h)
    y = norm.rms_norm_f64(h, w, EPS)
    assert np.all(np.abs(_f(v["y"]) - y) <= np.abs(y) * (2.0 ** -8 + 2.0 ** -20) + 2.0 ** -134)
    off = v["off"].cpu().numpy()
    rows = int(np.max(np.diff(off)))
    w13, w2 = _f(block["w13"]), _f(block["w2"])
    for name, f, args, Z, half in (
            ("c1", grouped.forward_f64, (_f(v["a"]), w13), H, 2.0 ** -8),
            ("c2", grouped.forward_f64, (_f(v["h1"]), w2), I, 2.0 ** -8),
            ("dh1", grouped.dgrad_f64, (_f(v["dc2"]), w2), H, 2.0 ** -8),
            ("da", grouped.dgrad_f64, (_f(v["dc1"]), w13), 2 * I, 2.0 ** -8),
            ("dw2", grouped.wgrad_f64, (_f(v["dc2"]), _f(v["h1b"])), rows, 2.0 ** -24),
            ("dw13", grouped.wgrad_f64, (_f(v["dc1"]), _f(v["a"])), rows, 2.0 ** -24)):
        _product(v[name], f(*args, off), f(*args, off, absolute=True), Z, half)
    dx, dw, mag, wmag = norm.rms_norm_backward_f64(h, w, _bits(v["dy"]), EPS, _bits(block["dout"]))
    assert np.all(np.abs(_f(v["dx"]) - dx) <= np.abs(dx) * 2.0 ** -8 + mag * 2.0 ** -19)
    assert np.all(np.abs(_f(v["dw"]) - dw) <= 11 * 2.0 ** -24 * wmag)
    n, c, outs = grouped.clip_f64([_f(v[k]) for k in ("dw13", "dw2", "drouter", "dw")], 0.5, 1e-6)
    assert abs(float(v["norm"]) - n) <= n * 2.0 ** -23 and c < 1.0
    for o, want in zip(v["clipped"], outs):
        assert np.all(np.abs(_f(o) - want) <= np.abs(want) * 2.0 ** -22 + 2.0 ** -134)
    q, s = fp4.quantize_mx(_bits(block["w13"]))
    assert np.array_equal(v["b13"].cpu().numpy(), q) and np.array_equal(v["sb13"].cpu().numpy(), s)
    A, SA = fp4.gather_mx(_bits(v["y"]), v["rows"].cpu().numpy(), K_TOP, T * K_TOP, v["a4"].cpu().numpy() * 0,
                          v["sa4"].cpu().numpy() * 0)
    assert np.array_equal(v["a4"].cpu().numpy(), A) and np.array_equal(v["sa4"].cpu().numpy(), SA)
    Af, Bf = fp4.decode_f64(A, SA, False), fp4.decode_f64(q, s, False)
    want, mag = grouped.forward_f64(Af, Bf, off), grouped.forward_f64(Af, Bf, off, absolute=True)
    err = fp32_sum_eps(H) * mag
    assert np.all(np.abs(_f(v["c4"]) - want) <= err + 2.0 ** -8 * (np.abs(want) + err))


def test_captured_and_replayed(gpu_lib, block):
    eager = _step(gpu_lib, block)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(gpu_lib, block)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(gpu_lib, block)
    flat = lambda d: [t for v in d.values() for t in (v if isinstance(v, list) else [v])]
    x0 = block["x"].clone()
    for i in range(4):
        for t in flat(got):
            t.zero_()
        block["x"].copy_(x0 if i != 2 else torch.roll(x0, 1, 0))     # other inputs in between
        graph.replay()
        torch.cuda.synchronize()
        want = eager if i != 2 else _step(gpu_lib, block)
        assert all(torch.equal(a, b) for a, b in zip(flat(got), flat(want))), i


def test_two_calls_at_a_time(gpu_lib, block):
    """The same step on two streams, each with its own outputs and workspaces."""
    want = _step(gpu_lib, block)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(_step(gpu_lib, block))
    torch.cuda.synchronize()
    for g in got:
        for k, t in want.items():
            assert all(torch.equal(a, b) for a, b in zip(g[k], t)) if isinstance(t, list) else torch.equal(g[k], t), k


def test_block_gradient_along_a_direction(gpu_lib, block):
    """dx . u and dW . u of the whole block against autograd in fp64 of the same function with the step's own routing.
    The step rounds to bf16 (2^-8) at nine places on the longest way back (y, a's product c1, h1, c2, the 8-bit copy
    of c1 with 2^-4, dc2, dh1, dc1, da, dy): the copy's rounding alone may move an element of dc1 by a few 2^-4, and
    relative to the gradient's norm the sum of independent roundings stays under 2^-4."""
    v = _step(gpu_lib, block)
    d = lambda t: t.double().cpu()
    x, w13, w2, w = (d(block[k]).requires_grad_() for k in ("x", "w13", "w2", "w"))
    router, res = d(block["router"]), d(block["res"])
    h = x + res
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w
    ids = v["ids"].cpu().long()
    l = (y @ router.t()).gather(1, ids)
    gw = torch.softmax(l, dim=1)
    out = h
    for j in range(K_TOP):
        c1 = torch.einsum("th,tnh->tn", y, w13[ids[:, j]])
        h1 = torch.nn.functional.silu(c1[:, :I]) * c1[:, I:]
        out = out + gw[:, j:j + 1] * torch.einsum("ti,thi->th", h1, w2[ids[:, j]])
    (out * d(block["dout"])).sum().backward()
    for got, want in ((v["dx"], x.grad), (v["dw13"], w13.grad), (v["dw2"], w2.grad), (v["dw"], w.grad)):
        g = d(got)
        assert float((g - want).norm()) <= 2.0 ** -4 * float(want.norm())
