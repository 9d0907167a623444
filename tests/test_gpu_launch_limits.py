"""Calls of more work items than one launch may have (2^32 threads a
dimension), within the documented limits: every output is written, and the
rows on both sides of a boundary are those of small calls.  Boundaries lie
at powers of two of tokens, slots or rows."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _need(gib):
    free = torch.cuda.mem_get_info()[0] >> 30
    if free < gib:
        pytest.skip(f"needs {gib} GiB of free device memory, {free} are free")


def _spots(T):
    """Short runs of rows at the start, around every power of two past 2^20, and at the end."""
    at = [0] + [1 << p for p in range(20, 31) if (1 << p) < T] + [T]
    return [(max(0, a - 3), min(T, a + 3)) for a in at]


def _finite_bf16(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-256, 257, (n,), generator=g, device="cuda", dtype=torch.int16).to(torch.bfloat16)


@pytest.mark.parametrize("T,E", [((1 << 27) + 3, 2), ((1 << 26) + 5, 33), ((1 << 26) + 3, 65)])
def test_gate(gpu_lib, T, E):
    _need(40)
    l = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    for a, b in _spots(T):
        l[a:b] = torch.randn((b - a, E), generator=torch.Generator().manual_seed(a % 1000)).to(torch.bfloat16).cuda()
    ids = torch.full((T, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), float("nan"), device="cuda")
    gpu_lib.topk_gate(l, 1, gpu_lib.GATE_SIGMOID, False, ids=ids, weights=w)
    assert int(ids.min()) == 0 and int(ids.max()) < E and float(w.min()) > 0
    d = torch.full_like(l, float("nan"))
    gpu_lib.topk_gate_backward(l, ids, w, gpu_lib.GATE_SIGMOID, False, out=d)
    assert not bool(torch.isnan(d.sum(dtype=torch.float32)))
    for a, b in _spots(T):
        i, v = gpu_lib.topk_gate(l[a:b].clone(), 1, gpu_lib.GATE_SIGMOID, False)
        assert torch.equal(ids[a:b], i) and torch.equal(w[a:b], v)
        assert torch.equal(d[a:b], gpu_lib.topk_gate_backward(l[a:b].clone(), i, v, gpu_lib.GATE_SIGMOID, False))


def test_dispatch(gpu_lib):
    T = (1 << 26) + 3
    x = _finite_bf16(T, 1).view(T, 1)
    rows = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    assert torch.equal(gpu_lib.dispatch(x, rows, 1, T), x.flip(0))


@pytest.mark.parametrize("T,K", [((1 << 24) + 3, 1), ((1 << 22) + 3, 1025)])
def test_dispatch_backward(gpu_lib, T, K):
    dA = _finite_bf16(T * K, 2).view(T, K)
    rows = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(gpu_lib.dispatch_backward(dA, rows, 1, out=out), dA.flip(0))


@pytest.mark.parametrize("T,k", [((1 << 25) + 3, 1), ((1 << 25) // 3 + 9, 3)])
def test_combine_backward(gpu_lib, T, k):
    C, dout = _finite_bf16(T * k, 3).view(-1, 1), _finite_bf16(T, 4).view(-1, 1)
    rows = torch.arange(T * k - 1, -1, -1, dtype=torch.int32, device="cuda")
    w = torch.randint(-4, 5, (T * k,), device="cuda").float()
    dC = torch.full_like(C, float("nan"))
    dw = torch.full_like(w, float("nan"))
    gpu_lib.combine_backward(C, dout, rows, w, k, dC=dC, dweights=dw)
    d = dout.float().repeat_interleave(k, dim=0)[:, 0]
    assert torch.equal(dw, C.float().flip(0)[:, 0] * d)
    assert torch.equal(dC[:, 0], (w * d).to(torch.bfloat16).flip(0))


def test_swiglu(gpu_lib):
    """Rows of 17 groups: two workgroups of 256 threads each."""
    _need(170)
    R, I = (1 << 23) + 3, 2176
    C = torch.zeros((R, 2 * I), dtype=torch.bfloat16, device="cuda")
    for a, b in _spots(R):
        C[a:b] = torch.randn((b - a, 2 * I), generator=torch.Generator().manual_seed(a % 1000)).to(torch.bfloat16).cuda()
    h, codes, scales = gpu_lib.swiglu(C, checkpoint=True)
    small = []
    for a, b in _spots(R):
        got = gpu_lib.swiglu(C[a:b].clone(), checkpoint=True)
        assert all(torch.equal(x, y[a:b]) for x, y in zip(got, (h, codes, scales)))
        small.append(got)
    assert float(scales[R // 3].sum()) == 34.0              # a row of zeros: its scales are 1
    del C
    dC = gpu_lib.swiglu_backward(codes, scales, h)
    for (a, b), (sh, sc, ss) in zip(_spots(R), small):
        assert torch.equal(dC[a:b], gpu_lib.swiglu_backward(sc, ss, sh))
