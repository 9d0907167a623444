"""The quantizing gather, SwiGLU with requantization and the combine at more
work items than one launch may have (2^32 threads): every output is written,
and the rows around every power of two are those of small calls."""

import pytest
import torch

pytestmark = pytest.mark.gpu

N = (1 << 26) + 3     # 64 threads each


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _spots():
    at = [0] + [1 << p for p in range(20, 27)] + [N]
    return [(max(0, a - 3), min(N, a + 3)) for a in at]


def _filled(width, gib):
    free = torch.cuda.mem_get_info()[0] >> 30
    if free < gib:
        pytest.skip(f"needs {gib} GiB of free device memory, {free} are free")
    x = torch.zeros((N, width), dtype=torch.bfloat16, device="cuda")
    for a, b in _spots():
        x[a:b] = torch.randn((b - a, width), generator=torch.Generator().manual_seed(a % 1000)).to(torch.bfloat16).cuda()
    return x


def _scales_of(SA, layout, a, b):
    return SA.view(1, N)[:, a:b] if layout else SA.view(N, 1)[a:b].t()


@pytest.mark.parametrize("layout", [0, 1])
def test_quantize_gather(gpu_lib, layout):
    x = _filled(128, 40)
    rows = torch.arange(N, dtype=torch.int32, device="cuda")
    A = torch.full((N, 128), 0x55, dtype=torch.uint8, device="cuda")
    SA = torch.full((N,), float("nan"), device="cuda")
    gpu_lib.quantize_gather(x, rows, 1, N, layout, A=A, SA=SA)
    assert not bool(torch.isnan(SA).any()) and not bool(A[N // 3].any()) and not bool(A[N - 100].any())
    for a, b in _spots():
        sA, sS = gpu_lib.quantize_gather(x[a:b].clone(), rows[: b - a].clone(), 1, b - a, layout)
        assert torch.equal(A[a:b], sA) and torch.equal(_scales_of(SA, layout, a, b).reshape(-1), sS.reshape(-1))


@pytest.mark.parametrize("layout", [0, 1])
def test_swiglu_quant(gpu_lib, layout):
    C = _filled(256, 60)
    A = torch.full((N, 128), 0x55, dtype=torch.uint8, device="cuda")
    SA = torch.full((N,), float("nan"), device="cuda")
    gpu_lib.swiglu_quant(C, layout, A=A, SA=SA)
    assert not bool(torch.isnan(SA).any()) and not bool(A[N // 3].any()) and not bool(A[N - 100].any())
    for a, b in _spots():
        sA, sS = gpu_lib.swiglu_quant(C[a:b].clone(), layout)
        assert torch.equal(A[a:b], sA) and torch.equal(_scales_of(SA, layout, a, b).reshape(-1), sS.reshape(-1))


def test_combine(gpu_lib):
    C = _filled(8, 10)
    rows = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = torch.full((N, 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(gpu_lib.combine(C, rows, torch.ones(N, device="cuda"), 1, out=out), C.flip(0))
