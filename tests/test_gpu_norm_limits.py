"""The norm of as many rows as its argument may name."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 4])
def test_as_many_rows_as_an_int_names(gpu_lib, T):
    """Several rows share a workgroup where they are short: T + 3 does not fit an int."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of free device memory")
    x = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    y = torch.full((T, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    spots = sorted({r for a in (0, 1 << 20, 1 << 25, 1 << 30, T) for r in range(max(0, a - 5), min(T, a + 5))})
    for r in spots:
        x[r] = 2.0 if r % 2 else -2.0
    gpu_lib.rms_norm(x, None, 12.0, out=y)              # 2 / sqrt(4 + 12)
    f = y.view(-1)
    assert sum(int(torch.count_nonzero(f[i:i + (1 << 30)])) for i in range(0, T, 1 << 30)) == len(spots)
    assert all(float(f[r]) == (0.5 if r % 2 else -0.5) for r in spots)
    del x, y, f
    torch.cuda.empty_cache()
