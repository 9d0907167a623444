"""Products of a few tokens with 4-bit weights on the GPU (w4a8_matvec)
against the fp64 oracle.

Bound per output: (K / 32 + 48) 2^-23 of the sum of its products' magnitudes
(INT4: of |x| (q + z + 32) s, since a product may be formed about an offset),
then half a bf16 unit: an fp32 sum in steps of at least 32 terms, each step
rounding at the size of the partial sums, and a few roundings for the group
scales and the join of the partial sums."""

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, matvec_f64

pytestmark = pytest.mark.gpu

MX, NV, INT4 = 0, 1, 2


def _problem(fmt, X, E, N, K, group, seed, zeros=True, gs=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((X, K), generator=g).to(torch.bfloat16)
    B = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    z = None
    if fmt == MX:
        SB = torch.randint(112, 132, (E, N, K // 32), generator=g, dtype=torch.int32).to(torch.uint8)
    elif fmt == NV:
        SB = torch.randint(0, 256, (E, N, K // 16), generator=g, dtype=torch.int32).to(torch.uint8)
        SB[(SB & 0x7F) == 0x7F] = 0x38
    else:
        SB = torch.randn((E, N, K // group), generator=g).to(torch.bfloat16)
        if zeros:
            z = torch.randint(0, 16, (E, N, K // group), generator=g, dtype=torch.int32).to(torch.uint8)
    s = torch.rand(E, generator=g) + 0.5 if gs else None
    return x, B, SB, z, s


def _half_ulp(v):
    _, p = np.frexp(np.abs(v))
    return np.ldexp(0.5, np.maximum(p - 8, -133))


def _check(lib, fmt, x, B, SB, z, s, ids, label):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = lib.matvec(dev(x), dev(B), dev(SB), fmt, expert_ids=dev(ids), expert_scales=dev(s), zeros=dev(z))
    xb = x.view(torch.int16).numpy().view(np.uint16)
    SBn = SB.view(torch.int16).numpy().view(np.uint16) if fmt == INT4 else SB.numpy()
    zn = None if z is None else z.numpy()
    ref, mag = matvec_f64(xb, B.numpy(), SBn, fmt, ids=None if ids is None else ids.numpy(),
                          gs=None if s is None else s.numpy(), zeros=zn)
    K = x.shape[1]
    if fmt == INT4:  # |x| (q + z + 32) |sc|, from all-positive weights
        mag, _ = matvec_f64((xb & 0x7FFF), B.numpy(), SBn & 0x7FFF, fmt,
                            ids=None if ids is None else ids.numpy(), gs=None if s is None else s.numpy(),
                            zeros=np.zeros_like(zn) if zn is not None else np.zeros(SBn.shape, np.uint8))
        top, _ = matvec_f64((xb & 0x7FFF), np.full_like(B.numpy(), 0xFF), SBn & 0x7FFF, fmt,
                            ids=None if ids is None else ids.numpy(), gs=None if s is None else s.numpy(),
                            zeros=np.zeros(SBn.shape, np.uint8))
        mag = mag + top * (48 / 15)
    got = bf16_bits_to_f64(y.view(torch.int16).cpu().numpy().view(np.uint16))
    acc = mag * (K / 32 + 48) * 2.0 ** -23
    bound = acc + _half_ulp(np.abs(ref) + acc)
    err = np.abs(got - ref)
    print(f"{label}: largest error / bound {(err / np.maximum(bound, 1e-300)).max():.3f}", flush=True)
    assert (err <= bound).all()
    return y


DENSE = [(1, 1, 32), (1, 16, 128), (1, 17, 160), (2, 31, 512), (3, 100, 96), (4, 64, 2048), (5, 257, 6144),
         (8, 48, 1024), (9, 33, 256), (16, 80, 4096), (17, 20, 608), (64, 50, 384), (1, 6144, 2048)]
FORMATS = [(MX, 32), (NV, 16), (INT4, 32), (INT4, 64), (INT4, 128)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("X,N,K", DENSE)
def test_dense(gpu_lib, fmt, group, X, N, K):
    K = max(group, K // max(32, group) * max(32, group))
    x, B, SB, z, s = _problem(fmt, X, 1, N, K, group, X * 31 + N)
    _check(gpu_lib, fmt, x, B, SB, z, s, None, f"dense fmt={fmt} group={group} X={X} N={N} K={K}")


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("T,k,per_slot,E,N,K", [
    (1, 8, False, 32, 96, 640), (1, 8, True, 32, 100, 512), (3, 8, False, 9, 63, 384), (8, 8, True, 32, 40, 256),
    (8, 8, False, 2, 48, 256), (64, 1, False, 5, 33, 128), (5, 3, True, 1, 130, 1152), (2, 6, False, 70, 16, 2304)])
def test_experts(gpu_lib, fmt, group, T, k, per_slot, E, N, K):
    x, B, SB, z, s = _problem(fmt, T * k if per_slot else T, E, N, K, group, T * 7 + N, zeros=T % 2 == 1, gs=k > 3)
    rng = np.random.default_rng(T + E)
    ids = torch.from_numpy(rng.integers(0, E, T * k).astype(np.int32))
    if T * k > 4:
        ids[2], ids[T * k - 1] = -1, E                     # slots without an expert
    y = _check(gpu_lib, fmt, x, B, SB, z, s, ids, f"experts fmt={fmt} group={group} T={T} k={k} E={E} N={N} K={K}")
    if T * k > 4:
        assert not y[2].any() and not y[T * k - 1].any()


@pytest.mark.parametrize("fmt,group", [(MX, 32), (NV, 16), (INT4, 128)])
@pytest.mark.parametrize("X,K", [(2, 32768), (1, 66048), (2, 131072), (3, 224)])
def test_long_and_short_rows(gpu_lib, fmt, group, X, K):
    """Rows of x that fill the LDS, that do not fit in it, and shorter than a step."""
    K = K // max(32, group) * max(32, group)
    x, B, SB, z, s = _problem(fmt, X, 1, 19, K, group, K % 1000)
    _check(gpu_lib, fmt, x, B, SB, z, s, None, f"dense fmt={fmt} group={group} X={X} N=19 K={K}")


def test_repeats_streams_and_expert_scale_default(gpu_lib):
    x, B, SB, z, _ = _problem(INT4, 4, 3, 50, 512, 64, 5)
    ids = torch.tensor([0, 2, 2, 1], dtype=torch.int32)
    c = [t.cuda() for t in (x, B, SB, ids, z)]
    a = gpu_lib.matvec(c[0], c[1], c[2], INT4, expert_ids=c[3], zeros=c[4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = gpu_lib.matvec(c[0], c[1], c[2], INT4, expert_ids=c[3], zeros=c[4], expert_scales=torch.ones(3).cuda())
    side.synchronize()
    assert torch.equal(a, b)
    # a slot's row does not depend on which other slots share the call
    for s in range(4):
        one = gpu_lib.matvec(c[0][s:s + 1].contiguous(), c[1], c[2], INT4, expert_ids=c[3][s:s + 1], zeros=c[4])
        assert (one[0].float() - a[s].float()).abs().max() <= 0.01 * a[s].float().abs().max()


@pytest.mark.parametrize("fmt", [MX, NV])
def test_nan_scales_and_extreme_scales(gpu_lib, fmt):
    """NaN codes reach their columns alone; E8M0 code 0 (2^-127) and NVFP4 subnormals count in full."""
    x, B, SB, _, _ = _problem(fmt, 2, 2, 40, 256, 0, 6)
    SB[0, 3, 1] = 0xFF if fmt == MX else 0x7F
    if fmt == MX:
        SB[1, :, 0] = 0
        SB[1, :20, 1:] = 0
    else:
        SB[1, :20] = SB[1, :20] & 0x87
    ids = torch.tensor([0, 1], dtype=torch.int32)
    y = gpu_lib.matvec(x.cuda(), B.cuda(), SB.cuda(), fmt, expert_ids=ids.cuda()).float().cpu()
    assert torch.isnan(y[0, 3]) and int(torch.isnan(y).sum()) == 1
    xb = x.view(torch.int16).numpy().view(np.uint16)
    SB[0, 3, 1] = 0x38
    ref, mag = matvec_f64(xb, B.numpy(), SB.numpy(), fmt, ids=ids.numpy())
    assert (np.abs(y[1].double().numpy() - ref[1]) <= _half_ulp(ref[1]) * 1.01 + mag[1] * 56 * 2.0 ** -23).all()


def test_infinite_activation(gpu_lib):
    """An infinity in x stays infinite or becomes NaN in its own row; the other rows are untouched."""
    for fmt, group in FORMATS:
        x, B, SB, z, _ = _problem(fmt, 3, 1, 32, 256, group, 7)
        want = gpu_lib.matvec(x.cuda(), B.cuda(), SB.cuda(), fmt, zeros=None if z is None else z.cuda())
        x[1, 17] = float("inf")
        got = gpu_lib.matvec(x.cuda(), B.cuda(), SB.cuda(), fmt, zeros=None if z is None else z.cuda())
        assert torch.equal(got[[0, 2]], want[[0, 2]]) and not torch.isfinite(got[1]).any()


def test_empty_and_refusals(gpu_lib):
    x, B, SB, z, s = (None if t is None else t.cuda() for t in _problem(INT4, 2, 2, 32, 128, 64, 8))
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert gpu_lib.matvec(x, B, SB, INT4, expert_ids=ids).shape == (0, 32)
    err = gpu_lib.W4A8Error
    with pytest.raises(err):
        gpu_lib.matvec(x, B, SB, INT4)                                                 # two experts, no ids
    with pytest.raises(err):
        gpu_lib.matvec(x, B, SB, INT4, expert_ids=torch.zeros(3, dtype=torch.int32, device="cuda"))  # 3 slots, 2 rows
    with pytest.raises(err):
        gpu_lib.matvec(x, B, SB, INT4, expert_ids=torch.zeros(66, dtype=torch.int32, device="cuda"))
    with pytest.raises(err):
        gpu_lib.matvec(x, B, SB.to(torch.uint8), 3, expert_ids=ids)                    # unknown format
    with pytest.raises(TypeError):
        gpu_lib.matvec(x, B, SB.to(torch.uint8), INT4, expert_ids=ids)                 # scales of another type
    with pytest.raises(ValueError):
        gpu_lib.matvec(x[:, :64].contiguous(), B, SB, INT4, expert_ids=ids)            # K differs
    with pytest.raises(ValueError):
        gpu_lib.matvec(x, B, SB, INT4, expert_ids=ids, zeros=z[:1])
    with pytest.raises(TypeError):
        gpu_lib.matvec(x.float(), B, SB, INT4, expert_ids=ids)
