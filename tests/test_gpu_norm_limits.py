"""The norm of as many rows as its argument may name, and long sums of the weight
gradient.

The weight gradient's bound: a workgroup's part is an fp32 sum of ceil(T / 512)
products, one rounding each (2^-24 of the magnitudes' sum), of an xh off by
2^-21; the parts are added in 64 bits and rounded once: (ceil(T / 512) + 10)
2^-24 of the magnitudes' sum."""

import numpy as np
import pytest
import torch

from oracle import bf16_rne_bits, norm

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


@pytest.mark.parametrize("T,K", [(16384, 64), (16383, 200), (5000, 33), (40000, 8)])
def test_weight_gradient_over_many_rows(gpu_lib, T, K):
    rng = np.random.default_rng(T + K)
    h, dy = bf16_rne_bits(rng.standard_normal((T, K))), bf16_rne_bits(rng.standard_normal((T, K)))
    dev = lambda b: torch.from_numpy(b.view(np.int16).copy()).view(torch.bfloat16).cuda()
    _, dw, _, wmag = norm.rms_norm_backward_f64(h, None, dy, 1e-5)
    _, got = gpu_lib.rms_norm_backward(dev(h), None, dev(dy), 1e-5)
    bound = (-(-T // 512) + 10) * 2.0 ** -24 * wmag + 2.0 ** -149
    assert np.max(np.abs(got.cpu().numpy() - dw) / bound) <= 1.0
