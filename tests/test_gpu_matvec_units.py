"""w4a8_matvec where a workgroup takes several units of 16 columns: loads
that run on into the next unit, the accumulators' reset, the joins' two
buffers, shares that differ by one, waves without a step.  Against the fp64
oracle under the bound of test_gpu_matvec.py.

A launch has at most three workgroups per compute unit, 768 on 256 of them
(or one per slot, fewer), so more units than that give some workgroup two at
least."""

import numpy as np
import pytest
import torch

from test_gpu_matvec import FORMATS, INT4, MX, NV, _check, _problem

pytestmark = pytest.mark.gpu


def _several(units, label):
    most = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    assert units > most, f"{label}: {units} units, {most} workgroups"


ROUTED = [
    (8, 8, 4096, 512, 1),     # one slot per expert, two steps
    (8, 8, 4091, 640, 1),     # a short last step, ragged columns
    (24, 32, 6144, 256, 1),   # one step: three of four waves have none
    (16, 4, 6131, 512, 4),    # eight rows of an expert at once
    (64, 2, 16400, 512, 32),  # sixteen rows, two items per expert
    (12, 1, 16400, 1024, 12),
]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("S,E,N,K,each", ROUTED)
def test_routed(gpu_lib, fmt, group, S, E, N, K, each):
    label = f"S={S} E={E} N={N} K={K} fmt={fmt} group={group}"
    _several(min(S, E) * -(-N // 16), label)
    x, B, SB, z, s = _problem(fmt, S, E, N, K, group, S + N)
    rng = np.random.default_rng(S)
    ids = np.repeat(np.arange(E), each)[:S] if each > 1 else rng.permutation(E)[:S]
    ids = torch.from_numpy(rng.permutation(ids).astype(np.int32))
    assert len(ids) == S
    _check(gpu_lib, fmt, x, B, SB, z, s, ids, label)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("X,N,K", [(1, 24999, 256), (2, 16403, 512), (8, 16403, 640), (16, 16387, 512)])
def test_dense(gpu_lib, fmt, group, X, N, K):
    label = f"X={X} N={N} K={K} fmt={fmt} group={group}"
    _several(-(-N // 16), label)
    x, B, SB, z, s = _problem(fmt, X, 1, N, K, group, X + N)
    _check(gpu_lib, fmt, x, B, SB, z, s, None, label)


@pytest.mark.parametrize("fmt,group", [(MX, 32), (NV, 16), (INT4, 128)])
@pytest.mark.parametrize("E,slots", [(32, "one"), (32, "two"), (4, "skew")])
def test_many_slots_of_few_experts(gpu_lib, fmt, group, E, slots):
    """64 slots that all name one expert, two, or one far more often than the others."""
    S, N, K = 64, 1030, 512
    x, B, SB, z, s = _problem(fmt, S, E, N, K, group, E)
    rng = np.random.default_rng(E)
    ids = {"one": np.full(S, 5), "two": rng.choice([3, 30], S), "skew": np.where(rng.random(S) < 0.8, 1, rng.integers(0, 4, S))}
    _check(gpu_lib, fmt, x, B, SB, z, s, torch.from_numpy(ids[slots].astype(np.int32)),
           f"fmt={fmt} group={group} E={E} {slots}")
