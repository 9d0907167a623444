"""The grouped products with nearly 2^31 rows of one expert, where a row count and
a tile's size together pass 32 signed bits: forward, row gradient and weight
gradient (its sum over as many rows), widths of whole 16 bytes and below.  Rows
are zero but for short runs at both ends and around the powers of two, with
values whose products and sums are exact."""

import pytest
import torch

pytestmark = pytest.mark.gpu

R = 2_140_000_000   # 128-row tiles: R + 127 fits, R + the number of tiles does not


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _rows(off):
    at = [0, 1 << 20, 1 << 30, off[1], R]
    return sorted({r for a in at for r in range(max(0, a - 3), min(R, a + 3))})


def _nonzero(t):
    """Elements that are not zero, a part at a time (a mask of all of them would be as large as a product's rows)."""
    f = t.view(-1)
    return sum(int(torch.count_nonzero(f[i:i + (1 << 30)])) for i in range(0, f.numel(), 1 << 30))


@pytest.mark.parametrize("width", [8, 7])
@pytest.mark.parametrize("off", [[0, R, R], [0, R - 5, R]])
def test_as_many_rows_as_32_bits_hold(gpu_lib, width, off):
    torch.cuda.empty_cache()
    need = 2 * 2 * R * 8 + (4 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GiB of free device memory")
    A, C = (torch.zeros(R * width, dtype=torch.bfloat16, device="cuda").view(R, width) for _ in range(2))
    offsets = torch.tensor(off, dtype=torch.int32).cuda()
    W = torch.randint(1, 4, (2, width, width), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    spots = _rows(off)
    at_spots = lambda t: torch.stack([t[r] for r in spots]).float()
    values = torch.randint(1, 4, (len(spots), width), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    for r, v in zip(spots, values):
        A[r] = v
    expert = [int(r >= off[1]) for r in spots]
    want = torch.stack([values[i].float() @ W[e].float().t() for i, e in enumerate(expert)])
    gpu_lib.grouped_gemm_bf16(A, W, offsets, out=C)
    assert torch.equal(at_spots(C), want) and _nonzero(C) == want.numel()
    dW = gpu_lib.grouped_gemm_wgrad(A, C, offsets)
    sums = torch.zeros((2, width, width), device="cuda")
    for i, e in enumerate(expert):
        sums[e] += values[i].float()[:, None] * want[i][None, :]
    assert torch.equal(dW, sums)
    back = torch.stack([values[i].float() @ W[e].float() for i, e in enumerate(expert)])
    gpu_lib.grouped_gemm_dgrad(A, W, offsets, out=C)
    assert torch.equal(at_spots(C), back) and _nonzero(C) == back.numel()
