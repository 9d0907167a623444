"""The operators of a block whose experts are trained and then served in 4
bits, as cases to be measured.

Before the gate stands a root-mean-square norm with the residual's addition,
whose output the expert products read in bf16 or in 8 bits; trained experts
need the grouped products with bf16 weights and both of their gradients; their
gradients are clipped by one norm over all tensors; and the trained weights
are quantised to 4 bits and multiplied by activations in 4 bits.  `run`
computes each either in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, where `own` is true, through this package's
entry points.
"""

import math

import torch

own = False

DEV = "cuda"

# Sizes are those of this repository's workloads (synth/generate.py: 32
# experts top-8, hidden 6144, intermediate 2048; 12 experts top-8, 6144 x
# 3584; 64, 1152 and 16384 tokens) or near them, with odd token counts, odd
# widths, idle experts and unevenly filled ones among them.


def listed():
    return [
        # the norm before the experts of one decode step, 64 tokens, output in 8 bits: the smallest call
        dict(name="norm decode 8 bits", op="norm", T=64, K=6144, residual=True, out="m_major", w="bf16"),
        # the same norm over a prompt, output in bf16 for the router and bf16 experts
        dict(name="norm prompt", op="norm", T=16384, K=6144, residual=True, out="bf16", w="bf16"),
        # its gradient in a training step, the residual stream's gradient added on the way
        dict(name="norm backward", op="norm_bwd", T=16383, K=6144, dres=True, w="f32"),
        # gate/up products of a training step, 1152 tokens top-8, unevenly filled experts
        dict(name="experts forward", op="fwd", T=1152, k=8, E=32, N=4096, K=6144, skew=1.0, idle=0),
        # the same products of a decode step of 64 tokens: every expert's weights for a few rows
        dict(name="experts decode", op="fwd", T=64, k=8, E=12, N=6144, K=3584, skew=0.0, idle=0),
        # the rows' gradient, an odd batch, three experts idle
        dict(name="experts row gradient", op="dgrad", T=4095, k=8, E=32, N=4096, K=6144, skew=1.0, idle=3),
        # the down projection's weight gradient in fp32 over 16384 tokens: the largest case
        dict(name="experts weight gradient", op="wgrad", T=16384, k=8, E=32, N=6144, K=2048, skew=1.0, idle=0, out="f32"),
        # trained weights to NVFP4 and read back, as quantisation-aware steps do
        dict(name="weights to 4 bits NV", op="fp4", fmt="nv", E=12, N=6144, K=3584),
        # gate/up products of 4-bit rows and 4-bit weights, the large prefill of 16384 tokens
        dict(name="products 4 by 4 bits", op="a4", T=16384, k=8, E=32, N=4096, K=6144, skew=1.0, idle=0, quant=False),
        # bf16 tokens quantised into their grouped rows, then the product: a decode step
        dict(name="decode 4 by 4 bits", op="a4", T=64, k=8, E=32, N=4096, K=6144, skew=1.0, idle=0, quant=True),
        # clipping of a small trained block: many small tensors of any length, fp32 and bf16
        dict(name="clip small block", op="clip", kind="many", n=40, most=300000, max_norm=1.0),
        # clipping the gradients of two blocks of 12 experts, bf16
        dict(name="clip experts", op="clip", kind="blocks", layers=2, E=12, N=6144, K=3584, max_norm=1.0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Row widths: multiples of 8 mostly, any width now and then."""
    n = _logint(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "fwd", "fwd", "dgrad", "wgrad", "fp4", "a4", "a4", "clip"])
    if op in ("norm", "norm_bwd"):
        out = rng.choice(["bf16", "row_major", "m_major"])
        K = _width(rng, 64, 8192)
        if op == "norm" and out != "bf16":
            K = max(1, K // 128) * 128
        T = _logint(rng, 1, min(16384, 90_000_000 // K))
        if op == "norm":
            return dict(op=op, T=T, K=K, residual=rng.random() < 0.6, out=out, w=rng.choice(["bf16", "f32"]))
        return dict(op=op, T=T, K=K, dres=rng.random() < 0.6, w=rng.choice(["bf16", "f32"]))
    if op in ("fwd", "dgrad", "wgrad", "a4"):
        E = _logint(rng, 2, 64)
        k = rng.randint(1, min(E, 8))
        if op == "a4":
            N, K = max(1, _logint(rng, 32, 6144) // 32) * 32, max(1, _logint(rng, 128, 6144) // 128) * 128
        else:
            N, K = _width(rng, 32, 6144), _width(rng, 32, 6144)
        most = min(16384 * 8, 400_000_000_000 // (N * K), 200_000_000 // max(N, K))
        c = dict(op=op, T=_logint(rng, 1, max(1, most // k)), k=k, E=E, N=N, K=K, skew=rng.choice([0.0, 1.0, 2.0]),
                 idle=rng.choice([0, 0, min(3, E - k)]))
        if op == "wgrad":
            c["out"] = rng.choice(["bf16", "f32"])
        if op == "a4":
            c["quant"] = rng.random() < 0.5
        return c
    if op == "fp4":
        E = _logint(rng, 1, 32)
        K = max(1, _logint(rng, 32, 6144) // 32) * 32
        return dict(op=op, fmt=rng.choice(["mx", "nv"]), E=E, N=_logint(rng, 1, min(6144, 200_000_000 // (E * K))), K=K)
    n = rng.randint(1, 60)
    return dict(op=op, kind="many", n=n, most=_logint(rng, 10, 20_000_000), max_norm=rng.choice([0.5, 1.0, 1e6]))


# --- inputs ----------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _randn_bf16(g, scale, *shape):
    """N(0, scale) in bf16, drawn along the first dimension so that fp32 copies stay small."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    step = max(1, 200_000_000 // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        out[i:i + step] = _randn(g, *out[i:i + step].shape) * scale
    return out


def _route(g, c):
    """(counts per expert, the grouped row of each slot): top-k of N(0,1) logits with a preference per expert,
    the last `idle` experts closed."""
    T, k, E = c["T"], c["k"], c["E"]
    l = _randn(g, T, E) + c["skew"] * _randn(g, 1, E)
    if c["idle"]:
        l[:, E - c["idle"]:] = -math.inf
    ids = torch.topk(l, k, dim=1)[1].reshape(-1)
    order = torch.sort(ids, stable=True)[1]
    rows = torch.empty(T * k, dtype=torch.int64, device=DEV)
    rows[order] = torch.arange(T * k, device=DEV)
    return torch.bincount(ids, minlength=E), rows.to(torch.int32)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _e2m1_code(v):
    """Codes 0..15 of v on the E2M1 grid (0, .5, 1, 1.5, 2, 3, 4, 6), halves to the even code, past 6 to 6."""
    a = v.abs()
    code = torch.where(a <= 2.0, torch.round(a * 2.0), torch.where(a <= 4.0, torch.round(a) + 2.0, torch.round(a * 0.5) + 4.0))
    return code.clamp(max=7.0).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def _e2m1_value(code):
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    return torch.cat([mag, -mag])[code.int()]


def _mx_groups(x):
    """Per 32 of the last dimension: (codes 0..15, E8M0 codes): scale 2^(floor(log2 amax) - 2), 1 for a zero group."""
    xg = x.float().unflatten(-1, (-1, 32))
    a = xg.abs().amax(dim=-1)
    e = torch.where(a > 0, (torch.frexp(a)[1].int() - 3).clamp(-127, 127), torch.zeros_like(a, dtype=torch.int32))
    return _e2m1_code(torch.ldexp(xg, -e[..., None])).flatten(-2), (e + 127).to(torch.uint8)


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _mx_pack(x):
    code, scales = _mx_groups(x)
    return _pack(code), scales


def _clip_sizes(c):
    if c["kind"] == "blocks":
        return [s for _ in range(c["layers"]) for s in ((c["E"], c["N"], c["K"]), (c["E"], c["K"]), (c["K"],))]
    # lengths over the whole range, 1 and the largest among them
    frac = [(0.6180339887 * i) % 1.0 for i in range(c["n"] - 1)] + [1.0]
    return [(max(1, int(round(c["most"] ** f))),) for f in frac]


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    st = dict(c)
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    if op in ("norm", "norm_bwd"):
        T, K = c["T"], c["K"]
        st["w"] = (1.0 + 0.1 * _randn(g, K)).to(bf if c["w"] == "bf16" else f32)
        st["eps"] = 1e-5
        st["x"] = _randn_bf16(g, 1.0, T, K) * (0.5 + torch.rand((T, 1), generator=g, device=DEV)).to(bf)
        if op == "norm":
            st["res"] = _randn_bf16(g, 2.0, T, K) if c["residual"] else None
            st["sum"] = torch.empty((T, K), dtype=bf, device=DEV) if c["residual"] else None
            if c["out"] == "bf16":
                st["y"] = torch.empty((T, K), dtype=bf, device=DEV)
            else:
                st["A"] = torch.empty((T, K), dtype=u8, device=DEV)
                st["SA"] = torch.empty((T, K // 128) if c["out"] == "row_major" else (K // 128, T), dtype=f32, device=DEV)
        else:
            st["dy"] = _randn_bf16(g, 0.01, T, K)
            st["dh"] = _randn_bf16(g, 0.01, T, K) if c["dres"] else None
            st["dx"] = torch.empty((T, K), dtype=bf, device=DEV)
            st["dw"] = torch.empty(K, dtype=f32, device=DEV)
        return st
    if op in ("fwd", "dgrad", "wgrad", "a4"):
        E, N, K, R = c["E"], c["N"], c["K"], c["T"] * c["k"]
        counts, rows = _route(g, c)
        st["bounds"] = [0] + torch.cumsum(counts, 0).tolist()
        st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device=DEV)
        if op in ("fwd", "wgrad"):
            st["A"] = _randn_bf16(g, 1.0, R, K)
        if op in ("dgrad", "wgrad"):
            st["dC"] = _randn_bf16(g, 0.1, R, N)
        if op in ("fwd", "dgrad"):
            st["W"] = _randn_bf16(g, 0.02, E, N, K)
        if op == "a4":
            st["B"] = torch.empty((E, N, K // 2), dtype=u8, device=DEV)
            st["SB"] = torch.empty((E, N, K // 32), dtype=u8, device=DEV)
            for e in range(E):
                st["B"][e], st["SB"][e] = _mx_pack(0.02 * _randn(g, N, K))
            st["A4"] = torch.empty((R, K // 2), dtype=u8, device=DEV)
            st["SA4"] = torch.empty((R, K // 32), dtype=u8, device=DEV)
            if c["quant"]:
                st["x"], st["rows"] = _randn_bf16(g, 1.0, c["T"], K), rows
            else:
                for i in range(0, R, 8192):
                    st["A4"][i:i + 8192], st["SA4"][i:i + 8192] = _mx_pack(_randn(g, min(8192, R - i), K))
        shape = (R, K) if op == "dgrad" else (E, N, K) if op == "wgrad" else (R, N)
        st["out"] = torch.empty(shape, dtype=f32 if c.get("out") == "f32" else bf, device=DEV)
        return st
    if op == "fp4":
        E, N, K = c["E"], c["N"], c["K"]
        st["W"] = _randn_bf16(g, 0.02, E, N, K)
        st["B"] = torch.empty((E, N, K // 2), dtype=u8, device=DEV)
        st["SB"] = torch.empty((E, N, K // (32 if c["fmt"] == "mx" else 16)), dtype=u8, device=DEV)
        st["gs"] = torch.empty(E, dtype=f32, device=DEV) if c["fmt"] == "nv" else None
        st["back"] = torch.empty((E, N, K), dtype=bf, device=DEV)
        return st
    if op == "clip":
        st["grads"] = []
        for i, s in enumerate(_clip_sizes(c)):
            t = _randn_bf16(g, 0.01, *s)
            st["grads"].append(t.float() if (len(s) < 3 and i % 3 != 1) else t)
        st["out"] = [torch.empty_like(t) for t in st["grads"]]
        st["norm"] = torch.empty(1, dtype=f32, device=DEV)
        return st
    raise ValueError(op)


# --- one pass --------------------------------------------------------------


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import moe_grouped_precision_amd as w4a8

    op = st["op"]
    if op == "norm":
        if st["out"] == "bf16":
            r = w4a8.rms_norm(st["x"], st["w"], st["eps"], residual=st["res"], out=st["y"], sum_out=st["sum"])
            return {"y": r[0], "sum": r[1]} if st["residual"] else r
        layout = w4a8.SCALE_ROW_MAJOR if st["out"] == "row_major" else w4a8.SCALE_M_MAJOR
        r = w4a8.rms_norm_quant(st["x"], st["w"], layout, st["eps"], residual=st["res"], A=st["A"], SA=st["SA"],
                                sum_out=st["sum"])
        got = {"codes": r[0].view(torch.float8_e4m3fn), "scales": r[1]}
        return {**got, "sum": r[2]} if st["residual"] else got
    if op == "norm_bwd":
        dx, dw = w4a8.rms_norm_backward(st["x"], st["w"], st["dy"], st["eps"], dh=st["dh"], dx=st["dx"],
                                        dweight=st["dw"])
        return {"dx": dx, "dw": dw}
    if op == "fwd":
        return w4a8.grouped_gemm_bf16(st["A"], st["W"], st["offsets"], out=st["out"])
    if op == "dgrad":
        return w4a8.grouped_gemm_dgrad(st["dC"], st["W"], st["offsets"], out=st["out"])
    if op == "wgrad":
        return w4a8.grouped_gemm_wgrad(st["dC"], st["A"], st["offsets"], out=st["out"])
    if op == "a4":
        if st["quant"]:
            w4a8.quantize_gather_fp4(st["x"], st["rows"], st["k"], st["T"] * st["k"], A=st["A4"], SA=st["SA4"])
        return w4a8.grouped_gemm_a4(st["A4"], st["SA4"], st["B"], st["SB"], st["offsets"], out=st["out"])
    if op == "fp4":
        fmt = w4a8.WSCALE_MX if st["fmt"] == "mx" else w4a8.WSCALE_NV
        B, SB, gs = w4a8.quantize_fp4(st["W"], fmt, B=st["B"], SB=st["SB"], expert_scales=st["gs"])
        return w4a8.dequantize_fp4(B, SB, fmt, expert_scales=gs, out=st["back"])
    norm = w4a8.clip_grads(st["grads"], st["max_norm"], out=st["out"], norm=st["norm"])
    return {"norm": norm, "grads": st["out"]}


def _norm_parts(h, eps):
    hf = h.float()
    return hf, 1.0 / torch.sqrt((hf * hf).mean(1, keepdim=True) + eps)


def _mx_values(codes, scales):
    """Packed MXFP4 [.., K/2] and E8M0 [.., K/32] -> fp32 values [.., K]."""
    q = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    return (_e2m1_value(q).unflatten(-1, (-1, 32)) * _pow2(scales.int() - 127)[..., None]).flatten(-2)


def _run_plain(st):
    op = st["op"]
    bf = torch.bfloat16
    if op == "norm":
        h = (st["x"].float() + st["res"].float()).to(bf) if st["residual"] else st["x"]
        hf, inv = _norm_parts(h, st["eps"])
        y = hf * inv * st["w"].float()
        if st["out"] == "bf16":
            return {"y": y.to(bf), "sum": h} if st["residual"] else y.to(bf)
        yg = y.unflatten(1, (-1, 128))
        a = yg.abs().amax(dim=2)
        s = torch.where(a > 0, a / torch.full_like(a, 448.0), torch.ones_like(a))
        q = (yg * (torch.ones_like(s) / s)[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).flatten(1)
        got = {"codes": q, "scales": s if st["out"] == "row_major" else s.t().contiguous()}
        return {**got, "sum": h} if st["residual"] else got
    if op == "norm_bwd":
        hf, inv = _norm_parts(st["x"], st["eps"])
        xh, dy = hf * inv, st["dy"].float()
        d = dy * st["w"].float()
        dx = inv * (d - xh * (d * xh).mean(1, keepdim=True))
        if st["dres"]:
            dx = dx + st["dh"].float()
        return {"dx": dx.to(bf), "dw": (dy * xh).sum(0)}
    if op in ("fwd", "dgrad", "wgrad", "a4"):
        b = st["bounds"]
        out = torch.zeros_like(st["out"])
        if op == "a4":
            A4, SA4 = st["A4"], st["SA4"]
            if st["quant"]:
                q, s = _mx_pack(st["x"])
                at = torch.arange(st["T"] * st["k"], device=q.device) // st["k"]
                A4, SA4 = torch.empty_like(A4), torch.empty_like(SA4)
                A4[st["rows"].long()], SA4[st["rows"].long()] = q[at], s[at]
        for e in range(st["E"]):
            r = slice(b[e], b[e + 1])
            if op == "fwd":
                out[r] = st["A"][r].float() @ st["W"][e].float().t()
            elif op == "dgrad":
                out[r] = st["dC"][r].float() @ st["W"][e].float()
            elif op == "wgrad":
                out[e] = st["dC"][r].float().t() @ st["A"][r].float()
            else:
                out[r] = _mx_values(A4[r], SA4[r]) @ _mx_values(st["B"][e], st["SB"][e]).t()
        return out
    if op == "fp4":
        if st["fmt"] == "mx":
            return _mx_values(*_mx_pack(st["W"])).to(bf)
        # bf16 weights meet the borders of both grids often: the decisions are taken in 64 bits
        x = st["W"].float().unflatten(2, (-1, 16))
        a = x.abs().amax(dim=3)
        gs = a.amax(dim=(1, 2))
        gs = torch.where(gs > 0, gs / torch.full_like(gs, 6.0 * 448.0), torch.ones_like(gs)).double()
        out = torch.empty_like(st["back"])
        for i in range(st["E"]):
            r = a[i].double() / (6.0 * gs[i])
            u = torch.exp2(torch.clamp(torch.floor(torch.log2(r)), min=-6.0) - 3.0)
            s = torch.round(r / u) * u
            t = (s * gs[i])[..., None]
            v = x[i].double() / torch.where(t > 0, t, torch.full_like(t, math.inf))
            out[i] = (_e2m1_value(_e2m1_code(v)) * t).flatten(1).to(bf)
        return out
    norm = torch.sqrt(sum((t.float() ** 2).sum(dtype=torch.float64) for t in st["grads"]))
    coef = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0).float()
    return {"norm": norm.float().view(1), "grads": [(t.float() * coef).to(t.dtype) for t in st["grads"]]}


# --- the definitions in 64 bits --------------------------------------------


def _grid(y, man, emin, most):
    """y on a floating grid of `man` mantissa bits whose smallest normal binade starts at 2^emin, halves to even."""
    e = torch.clamp(torch.frexp(y.abs())[1] - 1, min=emin)
    step = torch.ldexp(torch.ones_like(y), e - man)
    return torch.clamp(torch.round(y / step) * step, -most, most)


def _exact_mx(x):
    """MXFP4's values of x in 64 bits (floor of log2 by frexp)."""
    b = x.to(torch.float64).unflatten(-1, (-1, 32))
    a = torch.linalg.vector_norm(b, ord=math.inf, dim=-1, keepdim=True)
    s = torch.ldexp(torch.ones_like(a), torch.frexp(a)[1] - 3)
    s = torch.where(a > 0, s, torch.ones_like(s))
    return (_grid(b / s, 1, 0, 6.0) * s).flatten(-2)


def _decode_mx(codes, scales):
    c = codes.to(torch.int32)
    q = torch.empty((*c.shape[:-1], c.shape[-1] * 2), dtype=torch.int32, device=c.device)
    q[..., 0::2] = c % 16
    q[..., 1::2] = torch.div(c, 16, rounding_mode="floor")
    ex, man = (q >> 1) & 3, (q & 1).to(torch.float64)
    v = torch.where(ex == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, ex - 1))
    v = torch.where(q >= 8, -v, v)
    s = torch.ldexp(torch.ones(scales.shape, dtype=torch.float64, device=c.device), scales.to(torch.int32) - 127)
    return v * s.repeat_interleave(32, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    f64 = torch.float64
    if op == "norm":
        # the sum is rounded to bf16 where it is the residual stream; the norm is of what the stream holds
        h = (st["x"].to(f64) + st["res"].to(f64)).to(torch.bfloat16) if st["residual"] else st["x"]
        x = h.to(f64)
        y = x / torch.sqrt(torch.linalg.vecdot(x, x)[:, None] / st["K"] + st["eps"]) * st["w"].to(f64)
        if st["out"] == "bf16":
            return {"y": y, "sum": x} if st["residual"] else y
        b = y.unflatten(1, (-1, 128))
        s = torch.linalg.vector_norm(b, ord=math.inf, dim=2) / 448.0
        s = torch.where(s > 0, s, torch.ones_like(s))
        got = {"codes": _grid(b / s.unsqueeze(2), 3, -6, 448.0).flatten(1), "scales": s if st["out"] == "row_major" else s.t()}
        return {**got, "sum": x} if st["residual"] else got
    if op == "norm_bwd":
        x, dy, w = st["x"].to(f64), st["dy"].to(f64), st["w"].to(f64)
        n = torch.sqrt(torch.linalg.vecdot(x, x)[:, None] / st["K"] + st["eps"])
        # y = w x / n, n' = x / (K n): the chain rule written out
        dx = dy * w / n - x * torch.linalg.vecdot(dy * w, x)[:, None] / (st["K"] * n ** 3)
        if st["dres"]:
            dx = dx + st["dh"].to(f64)
        return {"dx": dx, "dw": torch.matmul(torch.ones((1, st["T"]), dtype=f64, device=DEV), dy * (x / n))[0]}
    if op in ("fwd", "dgrad", "wgrad", "a4"):
        out = torch.zeros(st["out"].shape, dtype=f64, device=DEV)
        which = torch.bucketize(torch.arange(st["T"] * st["k"], device=DEV), st["offsets"][1:].long(), right=True)
        xq = _exact_mx(st["x"]) if op == "a4" and st["quant"] else None
        for e in torch.unique(which).tolist():
            r = torch.nonzero(which == e)[:, 0]
            if op == "fwd":
                out[r] = torch.matmul(st["A"][r].to(f64), st["W"][e].to(f64).t().contiguous())
            elif op == "dgrad":
                out[r] = torch.matmul(st["dC"][r].to(f64), st["W"][e].to(f64))
            elif op == "wgrad":
                out[e] = torch.matmul(st["dC"][r].to(f64).t().contiguous(), st["A"][r].to(f64))
            else:
                if xq is not None:
                    slot = torch.argsort(st["rows"].long())[r]
                    a = xq[torch.div(slot, st["k"], rounding_mode="floor")]
                else:
                    a = _decode_mx(st["A4"][r], st["SA4"][r])
                out[r] = torch.matmul(a, _decode_mx(st["B"][e], st["SB"][e]).t().contiguous())
        return out
    if op == "fp4":
        out = torch.empty(st["W"].shape, dtype=f64, device=DEV)
        for e in range(st["E"]):
            if st["fmt"] == "mx":
                out[e] = _exact_mx(st["W"][e])
                continue
            b = st["W"][e].to(f64).unflatten(1, (-1, 16))
            a = torch.linalg.vector_norm(b, ord=math.inf, dim=2)
            gs = (a.max() / 2688.0).float().to(f64)  # the format holds it in 32 bits
            s = _grid(a / (6.0 * gs), 3, -6, 448.0) * gs if float(gs) > 0 else a
            s = s.unsqueeze(2)
            out[e] = torch.where(s > 0, _grid(b / torch.where(s > 0, s, torch.ones_like(s)), 1, 0, 6.0) * s, torch.zeros_like(b)).flatten(1)
        return out
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.to(f64)) ** 2) for t in st["grads"]))
    c = min(1.0, st["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=f64, device=DEV), "grads": [t.to(f64) * c for t in st["grads"]]}


# --- what a pass cannot do without -----------------------------------------


def work(case):
    c = case
    op = c["op"]
    if op == "norm":
        n = c["T"] * c["K"]
        out = 2 * n if c["out"] == "bf16" else n + n // 32
        return {"bytes": 2 * n + (4 * n if c["residual"] else 0) + out, "flops": 5 * n}
    if op == "norm_bwd":
        n = c["T"] * c["K"]
        return {"bytes": n * (6 + (2 if c["dres"] else 0)) + 6 * c["K"], "flops": 12 * n}
    if op in ("fwd", "dgrad", "wgrad", "a4"):
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        R, open_ = T * k, E - c["idle"]
        D = open_ * (1.0 - (1.0 - k / open_) ** T)  # experts with a row, on average of an even routing
        fl = 2 * R * N * K
        if op == "a4":
            rows = 2 * T * K if c["quant"] else R * K * (1 / 2 + 1 / 32)
            return {"bytes": D * N * K * (1 / 2 + 1 / 32) + rows + 2 * R * N, "flops": fl}
        if op == "wgrad":
            return {"bytes": 2 * R * (N + K) + E * N * K * (4 if c["out"] == "f32" else 2), "flops": fl}
        return {"bytes": 2 * D * N * K + 2 * R * (N + K), "flops": fl}
    if op == "fp4":
        n = c["E"] * c["N"] * c["K"]
        per = 1 / 2 + (1 / 32 if c["fmt"] == "mx" else 1 / 16)
        return {"bytes": n * (2 + per + 2), "flops": 4 * n}
    sizes = _clip_sizes(c)
    n = sum(math.prod(s) * (4 if (len(s) < 3 and i % 3 != 1) else 2) for i, s in enumerate(sizes))
    return {"bytes": 2 * n, "flops": 3 * sum(math.prod(s) for s in sizes)}
