"""The operators around the expert products, as cases to be measured.

An MoE block needs, next to the grouped products: the router's top-k gate and
its gradient; tokens moved to the experts' rows and back, with the gradients
of both moves; products of single tokens with 4-bit expert weights; and
SwiGLU that keeps its input in 8 bits for the backward pass.  `run` computes
each either in its plain form (elementary torch operations in 32 bits, one
rounding at the end) or, where `own` is true, through this package's entry
points.
"""

import math

import torch

own = False

DEV = "cuda"

# Sizes are those of this repository's workloads (synth/generate.py: 32
# experts top-8, hidden 6144, intermediate 2048; 12 experts top-8, 6144 x
# 3584; pools of 2048 and 6144 experts; 64, 1152 and 16384 tokens) or near
# them, with odd token counts, odd widths and masked slots among them.


def listed():
    return [
        # the router of one decode step: 64 tokens, 32 experts, the smallest call
        dict(name="gate decode", op="gate", T=64, E=32, k=8, dtype="f32", score="softmax", renorm=True),
        # the router over a wide shared pool (6144 experts), prompts of 2047 tokens
        dict(name="gate wide pool", op="gate", T=2047, E=6144, k=8, dtype="bf16", score="sigmoid", renorm=True),
        # the router's gradient in a training step of 16384 tokens, probabilities over all experts
        dict(name="gate backward", op="gate_bwd", T=16384, E=32, k=8, dtype="f32", score="softmax", renorm=False),
        # tokens to expert rows before the products, the large prefill: the largest case
        dict(name="dispatch prefill", op="dispatch", T=16384, k=8, K=6144, drop=0.0),
        # its gradient at 1151 tokens, some slots dropped by the router's mask
        dict(name="dispatch backward", op="dispatch_bwd", T=1151, k=8, K=6144, drop=0.05),
        # gradient of the weighted way back, 1152 tokens (the prefill down projection's output)
        dict(name="combine backward", op="combine_bwd", T=1152, k=8, N=6144, drop=0.02),
        # the same for a small ragged batch whose rows are not 16-byte multiples
        dict(name="combine backward odd", op="combine_bwd", T=37, k=3, N=1001, drop=0.2),
        # one new token, gate/up of its 8 of 32 experts, MXFP4
        dict(name="matvec one token MX", op="matvec", fmt="mx", T=1, k=8, per_slot=False, E=32, N=4096, K=6144,
             group=32, zeros=False),
        # three new tokens, down projection (each slot has its own row), NVFP4
        dict(name="matvec down NV", op="matvec", fmt="nv", T=3, k=8, per_slot=True, E=32, N=6144, K=2048,
             group=16, zeros=False),
        # a dense layer beside the experts, 5 new tokens, integer codes with zero points, ragged width
        dict(name="matvec dense int4", op="matvec", fmt="int4", T=5, k=0, per_slot=False, E=1, N=3583, K=6144,
             group=128, zeros=True),
        # SwiGLU of the gate/up output in a training step, input kept in 8 bits (1152 tokens top-8)
        dict(name="swiglu checkpoint", op="swiglu", R=9216, I=2048),
        # and its backward pass from the 8-bit copy, which also gives h back for the weight gradient
        dict(name="swiglu backward", op="swiglu_bwd", R=9215, I=2048),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Row widths: multiples of 8 mostly, any width now and then."""
    n = _logint(rng, lo, hi)
    return n if rng.random() < 0.35 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["gate", "gate_bwd", "dispatch", "dispatch_bwd", "combine_bwd", "matvec", "matvec", "swiglu",
                     "swiglu_bwd"])
    if op in ("gate", "gate_bwd"):
        E = _logint(rng, 4, 6144)
        T = _logint(rng, 1, min(16384, (1 << 25) // E))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 12)), dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5)
    if op in ("dispatch", "dispatch_bwd", "combine_bwd"):
        k = rng.randint(1, 10)
        w = _width(rng, 64, 8192)
        T = _logint(rng, 1, min(16384, 400_000_000 // (k * w)))
        return dict(op=op, T=T, k=k, drop=rng.choice([0.0, 0.02, 0.3]), **{"N" if op == "combine_bwd" else "K": w})
    if op == "matvec":
        fmt = rng.choice(["mx", "nv", "int4"])
        dense = rng.random() < 0.35
        k = 0 if dense else rng.randint(1, 8)
        T = _logint(rng, 1, 16 if dense else 64 // k)
        group = {"mx": 32, "nv": 16}.get(fmt) or rng.choice([32, 64, 128])
        step = max(32, group)
        K = max(1, _logint(rng, 256, 8192) // step) * step
        return dict(op=op, fmt=fmt, T=T, k=k, per_slot=bool(k) and rng.random() < 0.5, E=1 if dense else rng.randint(k, 32),
                    N=_width(rng, 64, 6144), K=K, group=group, zeros=fmt == "int4" and rng.random() < 0.5)
    R = _logint(rng, 1, 20000)
    return dict(op=op, R=R, I=128 * _logint(rng, 1, min(64, max(1, 40_000_000 // (128 * R)))))


# --- inputs ----------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    return g


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV, dtype=torch.float32)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _logits(g, c):
    """Router outputs: per-expert preferences plus N(0,1), some experts closed
    to a token (-inf), one token in 50 closed to all (padding)."""
    T, E = c["T"], c["E"]
    l = _randn(g, T, E) + _randn(g, 1, E)
    closed = _rand(g, T, E) < 0.1
    pad = _rand(g, T, 1) < 0.02
    l = torch.where(closed | pad, torch.full_like(l, -math.inf), l)
    return l.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)


def _select(l, k):
    """Ids of the k largest (ties to the lowest index), -1 where nothing is left."""
    v, i = torch.sort(l.float(), dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    ok = v != -math.inf
    return v, torch.where(ok, i, torch.full_like(i, -1)), ok


def _rows(g, T, k, drop, E=32):
    """The grouped row of each slot: a stable sort of the slots by expert, the
    dropped slots without a row (-1)."""
    ids = torch.randint(0, E, (T * k,), generator=g, device=DEV)
    ids = torch.where(_rand(g, T * k) < drop, torch.full_like(ids, E), ids)
    srt, order = torch.sort(ids, stable=True)
    rows = torch.empty(T * k, dtype=torch.int64, device=DEV)
    rows[order] = torch.arange(T * k, device=DEV)
    return torch.where(ids < E, rows, torch.full_like(rows, -1)).to(torch.int32)


def _e4m3_groups(x):
    """Per (row, 128): E4M3 values of x / s and s = amax / 448 (1 for a group below 2^-100)."""
    R, W = x.shape
    xg = x.float().view(R, W // 128, 128)
    a = xg.abs().amax(dim=2)
    s = torch.where(a < 2.0 ** -100, torch.ones_like(a), a / torch.full_like(a, 448.0))
    inv = torch.ones_like(s) / s
    return (xg * inv[:, :, None]).to(torch.float8_e4m3fn).view(R, W), s


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    st = dict(c)
    bf = torch.bfloat16
    if op in ("gate", "gate_bwd"):
        l = _logits(g, c)
        T, k = c["T"], c["k"]
        st["logits"], st["scale"] = l, 2.5
        if op == "gate":
            st["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
            st["w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        else:
            st["ids"] = _select(l, k)[1].to(torch.int32).contiguous()
            st["dw"] = _randn(g, T, k)
            st["out"] = torch.empty_like(l)
    elif op == "dispatch":
        T, k, K = c["T"], c["k"], c["K"]
        st["x"] = _randn(g, T, K).to(bf)
        st["rows"] = _rows(g, T, k, c["drop"])
        st["out"] = torch.zeros((T * k, K), dtype=bf, device=DEV)
    elif op == "dispatch_bwd":
        T, k, K = c["T"], c["k"], c["K"]
        st["dA"] = _randn(g, T * k, K).to(bf)
        st["rows"] = _rows(g, T, k, c["drop"])
        st["out"] = torch.empty((T, K), dtype=bf, device=DEV)
    elif op == "combine_bwd":
        T, k, N = c["T"], c["k"], c["N"]
        st["C"] = _randn(g, T * k, N).to(bf)
        st["dout"] = _randn(g, T, N).to(bf)
        st["rows"] = _rows(g, T, k, c["drop"])
        st["w"] = _rand(g, T * k)
        st["dC"] = torch.zeros((T * k, N), dtype=bf, device=DEV)
        st["dw"] = torch.empty(T * k, dtype=torch.float32, device=DEV)
    elif op == "matvec":
        T, k, E, N, K, grp = c["T"], c["k"], c["E"], c["N"], c["K"], c["group"]
        S = T * k if k else T
        X = S if c["per_slot"] else T
        st["S"], st["X"] = S, X
        st["x"] = _randn(g, X, K).to(bf)
        st["B"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        st["gs"] = st["z"] = None
        if c["fmt"] == "mx":
            st["SB"] = torch.randint(116, 124, (E, N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        elif c["fmt"] == "nv":
            st["SB"] = torch.randint(0x28, 0x58, (E, N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
            st["gs"] = 0.01 + 0.02 * _rand(g, E)
        else:
            st["SB"] = (0.002 + 0.02 * _rand(g, E, N, K // grp)).to(bf)
            if c["zeros"]:
                st["z"] = torch.randint(4, 12, (E, N, K // grp), generator=g, device=DEV, dtype=torch.uint8)
        st["ids"] = torch.argsort(_rand(g, T, E), dim=1)[:, :k].reshape(-1).to(torch.int32) if k else None
        st["out"] = torch.empty((S, N), dtype=bf, device=DEV)
    elif op == "swiglu":
        R, I = c["R"], c["I"]
        st["C"] = (_randn(g, R, 2 * I) * 1.5).to(bf)
        st["h"] = torch.empty((R, I), dtype=bf, device=DEV)
        st["codes"] = torch.empty((R, 2 * I), dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty((R, 2 * I // 128), dtype=torch.float32, device=DEV)
    elif op == "swiglu_bwd":
        R, I = c["R"], c["I"]
        q, s = _e4m3_groups((_randn(g, R, 2 * I) * 1.5).to(bf))
        st["codes"], st["scales"] = q.view(torch.uint8).contiguous(), s.contiguous()
        st["dh"] = _randn(g, R, I).to(bf)
        st["dC"] = torch.empty((R, 2 * I), dtype=bf, device=DEV)
        st["h"] = torch.empty((R, I), dtype=bf, device=DEV)
    else:
        raise ValueError(op)
    return st


# --- one pass --------------------------------------------------------------


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import moe_grouped_precision_amd as w4a8

    op = st["op"]
    if op in ("gate", "gate_bwd"):
        score = w4a8.GATE_SOFTMAX if st["score"] == "softmax" else w4a8.GATE_SIGMOID
        if op == "gate":
            ids, w = w4a8.topk_gate(st["logits"], st["k"], score, st["renorm"], st["scale"], ids=st["ids"],
                                    weights=st["w"])
            return {"ids": ids, "w": w}
        return w4a8.topk_gate_backward(st["logits"], st["ids"], st["dw"], score, st["renorm"], st["scale"],
                                       out=st["out"])
    if op == "dispatch":
        return w4a8.dispatch(st["x"], st["rows"], st["k"], st["T"] * st["k"], out=st["out"])
    if op == "dispatch_bwd":
        return w4a8.dispatch_backward(st["dA"], st["rows"], st["k"], out=st["out"])
    if op == "combine_bwd":
        dC, dw = w4a8.combine_backward(st["C"], st["dout"], st["rows"], st["w"], st["k"], dC=st["dC"],
                                       dweights=st["dw"])
        return {"dC": dC, "dw": dw}
    if op == "matvec":
        fmt = {"mx": w4a8.WSCALE_MX, "nv": w4a8.WSCALE_NV, "int4": w4a8.WSCALE_INT4}[st["fmt"]]
        return w4a8.matvec(st["x"], st["B"], st["SB"], fmt, expert_ids=st["ids"], expert_scales=st["gs"],
                           zeros=st["z"], out=st["out"])
    if op == "swiglu":
        h, codes, scales = w4a8.swiglu(st["C"], checkpoint=True, h=st["h"], codes=st["codes"], scales=st["scales"])
        return {"h": h, "codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    dC, h = w4a8.swiglu_backward(st["codes"], st["scales"], st["dh"], dC=st["dC"], h=st["h"])
    return {"dC": dC, "h": h}


def _gate_weights(v, ok, l, st):
    """The selected experts' weights before the scale, and the row maximum and sum of the softmax."""
    m = torch.where(ok[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))
    if st["score"] == "softmax":
        e = torch.exp(v - m)
        z = e.sum(1, keepdim=True) if st["renorm"] else torch.exp(l - m).sum(1, keepdim=True)
        w = e / z
    else:
        w = 1.0 / (1.0 + torch.exp(-v))
        if st["renorm"]:
            w = w / torch.where(ok, w, torch.zeros_like(w)).sum(1, keepdim=True)
    return torch.where(ok, w, torch.zeros_like(w)), m


def _run_plain(st):
    op = st["op"]
    if op == "gate":
        l = st["logits"].float()
        v, ids, ok = _select(l, st["k"])
        w, _ = _gate_weights(v, ok, l, st)
        return {"ids": ids.to(torch.int32), "w": w * st["scale"]}
    if op == "gate_bwd":
        l = st["logits"].float()
        ids = st["ids"].long()
        ok = ids >= 0
        at = ids.clamp(min=0)
        v = torch.where(ok, torch.gather(l, 1, at), torch.full_like(st["dw"], -math.inf))
        w, m = _gate_weights(v, ok, l, st)
        gr = torch.where(ok, st["dw"] * st["scale"], torch.zeros_like(st["dw"]))
        T, E = l.shape
        put = torch.where(ok, ids, torch.full_like(ids, E))  # a column past the last for what has no expert
        if st["score"] == "softmax" and not st["renorm"]:
            e = torch.exp(l - m)
            p = torch.where(ok[:, :1], e / e.sum(1, keepdim=True), torch.zeros_like(l))
            G = torch.zeros((T, E + 1), device=l.device).scatter_(1, put, gr)[:, :E]
            d = p * (G - (gr * w).sum(1, keepdim=True))
        else:
            if st["score"] == "softmax":
                d = w * (gr - (gr * w).sum(1, keepdim=True))
            else:
                s = torch.where(ok, 1.0 / (1.0 + torch.exp(-v)), torch.zeros_like(v))
                d = w * (gr - (gr * w).sum(1, keepdim=True)) * (1.0 - s) if st["renorm"] else gr * s * (1.0 - s)
            d = torch.zeros((T, E + 1), device=l.device).scatter_(1, put, d)[:, :E]
        return d.to(st["logits"].dtype)
    if op == "dispatch":
        T, k = st["T"], st["k"]
        rows = st["rows"].long()
        put = torch.where(rows >= 0, rows, torch.full_like(rows, T * k))  # a row past the last for dropped slots
        A = torch.zeros((T * k + 1, st["K"]), device=rows.device)
        A[put] = st["x"].float()[torch.arange(T * k, device=rows.device) // k]
        return A[: T * k].to(torch.bfloat16)
    if op == "dispatch_bwd":
        T, k = st["T"], st["k"]
        rows = st["rows"].long()
        d = st["dA"].float()[rows.clamp(min=0)] * (rows >= 0)[:, None]
        return d.view(T, k, -1).sum(1).to(torch.bfloat16)
    if op == "combine_bwd":
        T, k = st["T"], st["k"]
        rows = st["rows"].long()
        ok = rows >= 0
        d = st["dout"].float()[torch.arange(T * k, device=rows.device) // k]
        dw = (st["C"].float()[rows.clamp(min=0)] * d).sum(1) * ok
        put = torch.where(ok, rows, torch.full_like(rows, T * k))
        dC = torch.zeros((T * k + 1, st["N"]), device=rows.device)
        dC[put] = d * st["w"][:, None]
        return {"dC": dC[: T * k].to(torch.bfloat16), "dw": dw}
    if op == "matvec":
        return _matvec_plain(st)
    I = st["I"]
    if op == "swiglu":
        g, u = st["C"][:, :I].float(), st["C"][:, I:].float()
        q, s = _e4m3_groups(st["C"])
        return {"h": (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16), "codes": q, "scales": s}
    R = st["R"]
    v = (st["codes"].view(torch.float8_e4m3fn).float().view(R, -1, 128) * st["scales"][:, :, None]).view(R, 2 * I)
    g, u, dh = v[:, :I], v[:, I:], st["dh"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    dC = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], dim=1)
    return {"dC": dC.to(torch.bfloat16), "h": (g * sg * u).to(torch.bfloat16)}


def _matvec_plain(st):
    ids, S, N, K, grp = st["ids"], st["S"], st["N"], st["K"], st["group"]
    pick = (lambda t: t[ids.long()]) if ids is not None else (lambda t: t)
    B = pick(st["B"])
    q = torch.stack([B & 15, B >> 4], dim=-1).view(B.shape[0], N, K)
    SB = pick(st["SB"])
    if st["fmt"] == "int4":
        z = pick(st["z"]).float() if st["z"] is not None else torch.full(SB.shape, 8.0, device=SB.device)
        W = (q.view(-1, N, K // grp, grp).float() - z[..., None]) * SB.float()[..., None]
    else:
        mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
        val = torch.cat([mag, -mag]).index_select(0, q.reshape(-1).int()).view(-1, N, K // grp, grp)
        s = torch.exp2(SB.float() - 127.0) if st["fmt"] == "mx" else SB.view(torch.float8_e4m3fn).float()
        W = val * s[..., None]
    W = W.view(-1, N, K)
    x = st["x"].float()
    if ids is None:
        y = x @ W[0].t()
    else:
        y = torch.bmm(W, x.repeat_interleave(S // st["X"], dim=0)[:, :, None])[:, :, 0]
    if st["gs"] is not None:
        y = y * (st["gs"][ids.long()][:, None] if ids is not None else st["gs"])
    return y.to(torch.bfloat16)


# --- the definitions in 64 bits, one slot or one column of slots at a time --


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    f64 = torch.float64
    if op in ("gate", "gate_bwd"):
        return _exact_gate(st)
    if op in ("dispatch", "dispatch_bwd", "combine_bwd"):
        T, k = st["T"], st["k"]
        rows = st["rows"].long().view(T, k)
        if op == "dispatch":
            A = torch.zeros(st["out"].shape, dtype=f64, device=DEV)
            for j in range(k):
                t = torch.nonzero(rows[:, j] >= 0)[:, 0]
                A.index_copy_(0, rows[t, j], st["x"][t].to(f64))
            return A
        if op == "dispatch_bwd":
            dx = torch.zeros((T, st["K"]), dtype=f64, device=DEV)
            for j in range(k):
                t = torch.nonzero(rows[:, j] >= 0)[:, 0]
                dx.index_add_(0, t, st["dA"][rows[t, j]].to(f64))
            return dx
        dC = torch.zeros(st["C"].shape, dtype=f64, device=DEV)
        dw = torch.zeros((T, k), dtype=f64, device=DEV)
        for j in range(k):
            t = torch.nonzero(rows[:, j] >= 0)[:, 0]
            r = rows[t, j]
            dC.index_copy_(0, r, st["dout"][t].to(f64) * st["w"].view(T, k)[t, j].to(f64)[:, None])
            dw[t, j] = torch.linalg.vecdot(st["C"][r].to(f64), st["dout"][t].to(f64))
        return {"dC": dC, "dw": dw.view(-1)}
    if op == "matvec":
        return _exact_matvec(st)
    I = st["I"]
    if op == "swiglu":
        x = st["C"].to(f64)
        h = x[:, :I] * torch.sigmoid(x[:, :I]) * x[:, I:]
        blocks = x.unflatten(1, (-1, 128))
        s = torch.linalg.vector_norm(blocks, ord=math.inf, dim=2) / 448.0
        s = torch.where(s * 448.0 < 2.0 ** -100, torch.ones_like(s), s)
        y = blocks / s.unsqueeze(2)
        # the E4M3 grid: steps of 2^(e - 3) in a binade that starts at 2^e, e >= -6, halves to even
        e = torch.clamp(torch.frexp(y.abs())[1] - 1, min=-6)
        step = torch.ldexp(torch.ones_like(y), e - 3)
        return {"h": h, "codes": (torch.round(y / step) * step).flatten(1), "scales": s}
    q = st["codes"].to(torch.int32)
    ex, man = (q >> 3) & 15, (q & 7).to(f64)
    val = torch.where(ex == 0, man * 2.0 ** -9, torch.ldexp(1.0 + man / 8.0, ex - 7))
    val = torch.where(q >= 128, -val, val) * st["scales"].to(f64).repeat_interleave(128, dim=1)
    g, u, dh = val[:, :I], val[:, I:], st["dh"].to(f64)
    s = torch.sigmoid(g)
    return {"dC": torch.cat([dh * u * (s + g * s * torch.sigmoid(-g)), dh * (g * s)], dim=1), "h": g * s * u}


def _exact_gate(st):
    l = st["logits"].to(torch.float64)
    T, E = l.shape
    k, scale = st["k"], st["scale"]
    if st["op"] == "gate":
        left = l.clone()
        ids = []
        for _ in range(k):
            v, i = left.max(dim=1)
            i = (left == v[:, None]).to(torch.uint8).argmax(dim=1)  # the first of equals
            ids.append(torch.where(v > -math.inf, i, torch.full_like(i, -1)))
            left.scatter_(1, i[:, None], -math.inf)
        ids = torch.stack(ids, dim=1)
    else:
        ids = st["ids"].long()
    sel = torch.zeros((T, E), dtype=torch.bool, device=DEV)
    for j in range(k):
        t = torch.nonzero(ids[:, j] >= 0)[:, 0]
        sel[t, ids[t, j]] = True
    # weights laid out over all experts, then taken at the ids
    if st["score"] == "softmax":
        dom = torch.where(sel, l, torch.full_like(l, -math.inf)) if st["renorm"] else l
        P = torch.nan_to_num(torch.softmax(dom, dim=1), nan=0.0)
    else:
        P = torch.sigmoid(l) * sel
        if st["renorm"]:
            P = P / P.sum(1, keepdim=True).clamp(min=1e-300)
    at = ids.clamp(min=0)
    if st["op"] == "gate":
        return {"ids": None, "w": torch.where(ids >= 0, P.gather(1, at), 0.0) * scale}
    G = torch.zeros_like(l)
    for j in range(k):
        t = torch.nonzero(ids[:, j] >= 0)[:, 0]
        G[t, ids[t, j]] += scale * st["dw"][t, j].to(torch.float64)
    if st["score"] == "softmax":
        return P * (G - (P * G).sum(1, keepdim=True))
    if st["renorm"]:
        return P * (G - (P * G).sum(1, keepdim=True)) * torch.sigmoid(-l)
    return torch.nan_to_num(G * torch.sigmoid(l) * torch.sigmoid(-l))


def _exact_matvec(st):
    S, N, K, grp, fmt = st["S"], st["N"], st["K"], st["group"], st["fmt"]
    f64 = torch.float64
    y = torch.zeros((S, N), dtype=f64, device=DEV)
    experts = st["ids"].tolist() if st["ids"] is not None else [0] * S
    seen = {}
    for s, e in enumerate(experts):
        seen.setdefault(e, []).append(s)
    for e, slots in seen.items():
        B = st["B"][e].to(torch.int32)
        q = torch.empty((N, K), dtype=torch.int32, device=DEV)
        q[:, 0::2] = B % 16
        q[:, 1::2] = torch.div(B, 16, rounding_mode="floor")
        sc = st["SB"][e]
        if fmt == "int4":
            z = st["z"][e].to(f64) if st["z"] is not None else torch.full((N, K // grp), 8.0, dtype=f64, device=DEV)
            W = (q.to(f64) - z.repeat_interleave(grp, dim=1)) * sc.to(f64).repeat_interleave(grp, dim=1)
        else:
            ex, man = (q >> 1) & 3, (q & 1).to(f64)
            W = torch.where(ex == 0, 0.5 * man, torch.ldexp(1.0 + 0.5 * man, ex - 1))
            W = torch.where(q >= 8, -W, W)
            c = sc.to(torch.int32)
            if fmt == "mx":
                sv = torch.ldexp(torch.ones_like(c, dtype=f64), c - 127)
            else:  # codes here are positive E4M3 normals and subnormals
                sv = torch.where(c < 8, c.to(f64) * 2.0 ** -9, torch.ldexp(1.0 + (c % 8).to(f64) / 8.0, (c >> 3) - 7))
            W = W * sv.repeat_interleave(grp, dim=1)
        xs = st["x"][[s // (S // st["X"]) for s in slots]].to(f64)
        out = torch.matmul(W, xs.t().contiguous()).t()
        y[slots] = out * (st["gs"][e].to(f64) if st["gs"] is not None else 1.0)
    return y


# --- what a pass cannot do without -----------------------------------------


def work(case):
    c = case
    op = c["op"]
    if op in ("gate", "gate_bwd"):
        b = 2 if c["dtype"] == "bf16" else 4
        n, s = c["T"] * c["E"], c["T"] * c["k"]
        return {"bytes": n * b + 8 * s, "flops": 4 * n} if op == "gate" else {"bytes": 2 * n * b + 8 * s, "flops": 6 * n}
    if op in ("dispatch", "dispatch_bwd", "combine_bwd"):
        T, k, w = c["T"], c["k"], c.get("K") or c.get("N")
        kept = T * k * (1.0 - c["drop"])
        if op == "dispatch":
            return {"bytes": 2 * w * (T + kept) + 4 * T * k, "flops": 0}
        if op == "dispatch_bwd":
            return {"bytes": 2 * w * (T + kept) + 4 * T * k, "flops": kept * w}
        return {"bytes": 2 * w * (T + 2 * kept) + 12 * T * k, "flops": 3 * kept * w}
    if op == "matvec":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        S = T * k if k else T
        X = S if c["per_slot"] else T
        D = E * (1.0 - (1.0 - k / E) ** T) if k else 1  # experts that some slot names, on average
        per = K / 2 + (K / c["group"]) * {"mx": 1, "nv": 1, "int4": 3 if c["zeros"] else 2}[c["fmt"]]
        return {"bytes": D * N * per + 2 * X * K + 2 * S * N, "flops": 2 * S * N * K}
    R, I = c["R"], c["I"]
    groups = 4 * R * 2 * I / 128
    if op == "swiglu":
        return {"bytes": R * I * (4 + 2 + 2) + groups, "flops": 12 * R * I}
    return {"bytes": R * I * (2 + 2 + 4 + 2) + groups, "flops": 16 * R * I}
