"""Products with 4-bit weights where fp32 overflows on the way or an operand
is infinite, against the fp64 definition: the largest and smallest MXFP4
scales, infinities and NaN in x, values of x near bf16's largest.

Finite outputs have the bound of test_gpu_matvec.py, (K / 32 + 48) 2^-23 of
the products' magnitudes (an fp32 sum) and half a bf16 unit; INT4 magnitudes
about the offset, as there.  An output past bf16's largest value is infinite,
and signs of infinities and places of NaN are the definition's."""

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, matvec_f64
from test_gpu_matvec import FORMATS, INT4, MX, NV, _half_ulp, _problem

pytestmark = pytest.mark.gpu

BF16_MAX = 3.3895313892515355e38


def _compare(lib, fmt, x, B, SB, z, s, ids, label):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = lib.matvec(dev(x), dev(B), dev(SB), fmt, expert_ids=dev(ids), expert_scales=dev(s), zeros=dev(z))
    bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    xb, SBn = bits(x), bits(SB) if fmt == INT4 else SB.numpy()
    rest = dict(ids=None if ids is None else ids.numpy(), gs=None if s is None else s.numpy())
    with np.errstate(all="ignore"):
        ref, mag = matvec_f64(xb, B.numpy(), SBn, fmt, zeros=None if z is None else z.numpy(), **rest)
        if fmt == INT4:   # |x| (q + z + 32) |sc|
            top, _ = matvec_f64(xb & 0x7FFF, np.full_like(B.numpy(), 0xFF), SBn & 0x7FFF, fmt,
                                zeros=np.zeros(SBn.shape, np.uint8), **rest)
            mag = top * (62 / 15)
    got = bf16_bits_to_f64(y.view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{label}: NaN in {np.isnan(got).sum()}, not {np.isnan(ref).sum()}"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), label
    fin = np.isfinite(ref)
    acc = mag[fin] * (x.shape[1] / 32 + 48) * 2.0 ** -23
    r, g = ref[fin], got[fin]
    over = np.abs(r) + acc >= BF16_MAX * (1 + 2.0 ** -9)      # may round to infinity
    bound = acc + _half_ulp(np.abs(r) + acc)
    with np.errstate(invalid="ignore"):
        ok = (np.abs(g - r) <= bound) | (over & (np.abs(g) >= BF16_MAX) & (np.sign(g) == np.sign(r)))
    print(f"{label}: {fin.sum()} finite, {inf.sum()} infinite, {np.isnan(ref).sum()} NaN, {(~ok).sum()} off", flush=True)
    assert ok.all()
    return got, ref


# one step, a short last step, shorter than a step, several units of several workgroups
SHAPES = [(3, 40, 512), (2, 33, 640), (2, 20, 128), (9, 48, 768), (1, 13000, 256)]


@pytest.mark.parametrize("X,N,K", SHAPES)
def test_largest_and_smallest_mx_scales(gpu_lib, X, N, K):
    """Codes 253 and 254: a weight is up to 6 * 2^127, past fp32, and x of
    2^-40 brings the sum back; codes 0 to 2 beside them.  Rows of x that are
    zero where the large codes are leave the small ones in the sum."""
    x, B, SB, _, s = _problem(MX, X, 1, N, K, 32, X + N)
    g = torch.Generator().manual_seed(K)
    x = (x.float() * 2.0 ** -40).to(torch.bfloat16)
    pick = torch.tensor([253, 254, 252, 251, 0, 1, 2, 127])
    SB[:, ::2] = pick[torch.randint(0, 8, SB[:, ::2].shape, generator=g)].to(torch.uint8)
    SB[0, 1, :] = 254
    SB[0, 3, 0] = 254
    SB[0, 3, 1:] = 1
    if X > 1:
        x[1, :32] = 0
    got, ref = _compare(gpu_lib, MX, x, B, SB, None, s, None, f"X={X} N={N} K={K}")
    assert np.isfinite(ref).all() and np.isfinite(got).all()


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("X,N,K", SHAPES)
def test_infinities_and_nan_in_x(gpu_lib, fmt, group, X, N, K):
    K = max(group, K // group * group)
    x, B, SB, z, s = _problem(fmt, X, 1, N, K, group, N + K)
    clean = gpu_lib.matvec(x.cuda(), B.cuda(), SB.cuda(), fmt, expert_scales=s.cuda(),
                           zeros=None if z is None else z.cuda())
    x[0, 17] = float("inf")
    if X > 1:
        x[1, K - 1] = float("-inf")
    if X > 2:
        x[2, 3], x[2, K - 5] = float("inf"), float("-inf")
    if X > 4:
        x[4, K // 2] = float("nan")
    got, _ = _compare(gpu_lib, fmt, x, B, SB, z, s, None, f"fmt={fmt} group={group} X={X} N={N} K={K}")
    keep = [r for r in range(X) if r not in (0, 1, 2, 4)]
    clean = bf16_bits_to_f64(clean.view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(got[keep], clean[keep])            # the other rows' bits


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_values_near_the_largest(gpu_lib, fmt, group):
    """|x| up to 2^127 with scales that bring the sum back into range: sums of
    x q leave fp32 before their scale, and so do (16 + q) x."""
    X, N, K = 3, 40, 512
    x, B, SB, z, _ = _problem(fmt, X, 1, N, K, group, 3)
    x = (torch.sign(x.float()) * 2.0 ** 127 * (1 + torch.rand(x.shape) * 0.9)).to(torch.bfloat16)
    gs = torch.full((1,), 2.0 ** -30)
    if fmt == MX:
        SB = torch.randint(80, 100, SB.shape).to(torch.uint8)
    elif fmt == NV:
        SB = SB & 0x87
    else:
        SB = (SB.float() * 2.0 ** -20).to(torch.bfloat16)
    _compare(gpu_lib, fmt, x, B, SB, z, gs, None, f"fmt={fmt} group={group}")


def test_infinity_among_experts(gpu_lib):
    """Routed slots, several units per workgroup: only the infinite row's slots change."""
    x, B, SB, z, _ = _problem(INT4, 4, 3, 4300, 512, 64, 11)
    ids = torch.tensor([0, 2, 2, 1, 0, -1, 1, 2], dtype=torch.int32)
    x[2, 100] = float("inf")
    _compare(gpu_lib, INT4, x, B, SB, z, None, ids, "experts")
