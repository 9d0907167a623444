"""The MoE block of examples/moe_block.py on the GPU, every operator in its
place: the decoding path against the grouped one, and the gradients of the
training path against torch's autograd in fp64 with the same experts, the
same selection and exact arithmetic.

The paths round to bf16 after every stage (a dozen roundings of 2^-9 on the
way to a gradient) and the backward pass reads SwiGLU's input from 8 bits
(2^-4 per element, random in sign): the 2-norm of the difference stays within
4e-2 of the gradient's, and 2e-2 forward."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block_example", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("E,H,I,k,T", [(4, 256, 128, 2, 24), (8, 512, 256, 3, 7), (3, 128, 128, 3, 33)])
def test_block_forward_backward_decode(gpu_lib, example, E, H, I, k, T):
    block = example.MoEBlock(E, H, I, k, seed=E)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    out = block.forward(x)
    dout = torch.randn((T, H), generator=g).to(torch.bfloat16).cuda()
    dx, drouter = block.backward(dout)
    ids = block.saved[2].long().cpu()

    W13 = torch.stack([example.decode_mxfp4(b, s) for b, s in zip(block.B13, block.SB13)]).double().cpu()
    W2 = torch.stack([example.decode_mxfp4(b, s) for b, s in zip(block.B2, block.SB2)]).double().cpu()
    xd = x.double().cpu().requires_grad_(True)
    router = block.router.double().cpu().requires_grad_(True)
    w = torch.softmax((xd @ router.t()).gather(1, ids), dim=1)
    y = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            c = W13[ids[t, j]] @ xd[t]
            y[t] = y[t] + w[t, j] * (W2[ids[t, j]] @ (torch.nn.functional.silu(c[:I]) * c[I:]))
    y.backward(dout.double().cpu())
    errs = _rel(out.cpu(), y.detach()), _rel(dx.cpu(), xd.grad), _rel(drouter.cpu(), router.grad)
    print(f"E={E} H={H} I={I} k={k} T={T}: forward {errs[0]:.2e} dx {errs[1]:.2e} drouter {errs[2]:.2e}", flush=True)
    assert errs[0] <= 2e-2 and errs[1] <= 4e-2 and errs[2] <= 4e-2

    few = x[: 64 // k].contiguous()
    assert _rel(block.decode(few).cpu(), y.detach()[: 64 // k]) <= 2e-2


def test_decode_in_a_graph(gpu_lib, example):
    """The decoding path captured once and replayed on changing tokens, with
    eager work between the replays."""
    block = example.MoEBlock(6, 512, 256, 4, seed=2)
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn((3, 512), generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    want = [block.decode(x).clone() for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.decode(x)
    for i in (1, 0, 2, 1):
        y.zero_()
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_router_learns(gpu_lib, example):
    teacher = example.MoEBlock(8, 256, 128, 2, seed=4)
    student = example.MoEBlock(8, 256, 128, 2, seed=4)
    g = torch.Generator().manual_seed(5)
    student.router = student.router + 0.5 * torch.randn((8, 256), generator=g).cuda() / 16
    x = torch.randn((64, 256), generator=g).to(torch.bfloat16).cuda()
    losses = example.train_router(student, x, teacher.forward(x).float(), steps=15, lr=20.0)
    print("losses", losses, flush=True)
    assert losses[-1] < 0.9 * losses[0]
