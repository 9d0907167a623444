"""A mixture-of-experts block with frozen MXFP4 experts and a trained router.

    python examples/moe_block.py [--tokens 64] [--steps 20]

Training: gate -> route prep -> dispatch -> grouped product -> SwiGLU (its
input kept in 8 bits) -> grouped product -> combine, and back: the gradients
of combine, SwiGLU, dispatch and gate.  The library multiplies by the experts
in the forward direction; the gradient through a frozen expert is a plain
product with its decoded weights here.

Decoding: a few tokens run through the same experts without any grouping, by
matrix-vector products.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_grouped_precision_amd as w4a8  # noqa: E402
from synth import quantize_mxfp4  # noqa: E402


def decode_mxfp4(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """codes uint8 [N, K/2], scales uint8 [N, K/32] -> bf16 [N, K] (exact)."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    value = torch.cat([mag, -mag])
    q = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(codes.shape[0], -1)
    w = value[q.int()].view(codes.shape[0], -1, 32) * torch.exp2(scales.float() - 127.0)[:, :, None]
    return w.view(codes.shape[0], -1).to(torch.bfloat16)


class MoEBlock:
    """E experts of hidden size H and intermediate size I, top_k of them per token."""

    def __init__(self, E: int, H: int, I: int, top_k: int, seed: int = 0, device: str = "cuda"):
        g = torch.Generator().manual_seed(seed)
        self.E, self.H, self.I, self.top_k = E, H, I, top_k
        self.router = (torch.randn((E, H), generator=g) / H ** 0.5).to(device)
        w13 = [quantize_mxfp4(torch.randn((2 * I, H), generator=g) / H ** 0.5) for _ in range(E)]
        w2 = [quantize_mxfp4(torch.randn((H, I), generator=g) / I ** 0.5) for _ in range(E)]
        self.B13, self.SB13 = (torch.stack(t).to(device) for t in zip(*w13))
        self.B2, self.SB2 = (torch.stack(t).to(device) for t in zip(*w2))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x bf16 [T, H] -> bf16 [T, H]; keeps what backward needs."""
        k, T = self.top_k, x.shape[0]
        logits = x.float() @ self.router.t()
        ids, weights = w4a8.topk_gate(logits, k)
        _, offsets, rows = w4a8.route_prep(ids, self.E)
        a = w4a8.dispatch(x, rows, k, T * k)
        c1 = w4a8.grouped_gemm_a16(a, self.B13, self.SB13, w4a8.WSCALE_MX, offsets)
        h, codes, scales = w4a8.swiglu(c1, checkpoint=True)
        c2 = w4a8.grouped_gemm_a16(h, self.B2, self.SB2, w4a8.WSCALE_MX, offsets)
        self.saved = (x, logits, ids, weights, offsets, rows, codes, scales, c2)
        return w4a8.combine(c2, rows, weights, k)

    def backward(self, dout: torch.Tensor):
        """dout bf16 [T, H] -> (dx bf16 [T, H], drouter fp32 [E, H])."""
        x, logits, ids, weights, offsets, rows, codes, scales, c2 = self.saved
        k = self.top_k
        dc2, dweights = w4a8.combine_backward(c2, dout, rows, weights, k)
        bounds = offsets.tolist()
        dh = torch.zeros((dc2.shape[0], self.I), dtype=torch.bfloat16, device=x.device)
        da = torch.zeros((dc2.shape[0], self.H), dtype=torch.bfloat16, device=x.device)
        for e in range(self.E):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                dh[lo:hi] = dc2[lo:hi] @ decode_mxfp4(self.B2[e], self.SB2[e])
        dc1 = w4a8.swiglu_backward(codes, scales, dh)
        for e in range(self.E):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                da[lo:hi] = dc1[lo:hi] @ decode_mxfp4(self.B13[e], self.SB13[e])
        dlogits = w4a8.topk_gate_backward(logits, ids, dweights)
        dx = w4a8.dispatch_backward(da, rows, k)
        return (dx.float() + dlogits @ self.router).to(torch.bfloat16), dlogits.t() @ x.float()

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """The same block for a few tokens (tokens * top_k at most 64)."""
        k = self.top_k
        ids, weights = w4a8.topk_gate(x.float() @ self.router.t(), k)
        slots = ids.view(-1)
        c1 = w4a8.matvec(x, self.B13, self.SB13, w4a8.WSCALE_MX, expert_ids=slots)
        c2 = w4a8.matvec(w4a8.swiglu(c1), self.B2, self.SB2, w4a8.WSCALE_MX, expert_ids=slots)
        rows = torch.arange(slots.numel(), dtype=torch.int32, device=x.device)
        return w4a8.combine(c2, rows, weights, k)


def train_router(block: MoEBlock, x: torch.Tensor, target: torch.Tensor, steps: int, lr: float):
    """Steps of gradient descent on the router alone; the losses.  A step that
    raised the loss (the selection changes in jumps) is taken back and the
    rate quartered."""
    losses, kept = [], None
    for _ in range(steps):
        err = block.forward(x).float() - target
        loss = float((err * err).mean())
        if kept is not None and loss > losses[-1]:
            block.router, drouter = kept
            lr *= 0.25
            losses.append(losses[-1])
        else:
            _, drouter = block.backward((2.0 / err.numel() * err).to(torch.bfloat16))
            kept = block.router, drouter
            losses.append(loss)
        block.router = block.router - lr * drouter
    block.router = kept[0]
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--intermediate", type=int, default=512)
    ap.add_argument("--top-k", type=int, default=2)
    a = ap.parse_args()
    teacher = MoEBlock(a.experts, a.hidden, a.intermediate, a.top_k, seed=1)
    student = MoEBlock(a.experts, a.hidden, a.intermediate, a.top_k, seed=1)
    student.router = student.router + 0.5 * torch.randn_like(student.router) / a.hidden ** 0.5
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    losses = train_router(student, x, teacher.forward(x).float(), a.steps, lr=20.0)
    print(f"router loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    few = x[: max(1, min(a.tokens, 64 // a.top_k, 4))].contiguous()
    for _ in range(3):
        y = student.decode(few)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(100):
        y = student.decode(few)
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) * 1e4
    diff = (y.float() - student.forward(few).float()).abs().max()
    print(f"decode of {few.shape[0]} tokens: {us:.1f} us, largest difference to the grouped path {diff:.2e}")


if __name__ == "__main__":
    main()
