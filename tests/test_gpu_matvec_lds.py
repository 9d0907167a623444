"""w4a8_matvec with more than 64 KB of LDS, which a kernel has to be allowed
first: two host threads that call one kernel with different amounts, and a
call inside a captured graph."""

import threading

import pytest
import torch

from test_gpu_matvec import FORMATS, MX, _problem

pytestmark = pytest.mark.gpu


def _case(fmt, X, N, K, group, seed):
    x, B, SB, z, s = _problem(fmt, X, 1, N, K, group, seed)
    kw = dict(expert_scales=s.cuda(), zeros=None if z is None else z.cuda())
    return (x.cuda(), B.cuda(), SB.cuda(), fmt), kw


def test_threads_with_different_amounts(gpu_lib):
    """16 rows of x in LDS, K = 2048 (about 100 KB) and 4096 (past 150 KB), the same kernel."""
    cases = [_case(MX, 16, 64, K, 32, K) for K in (2048, 4096)]
    want = [gpu_lib.matvec(*a, **kw) for a, kw in cases]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        a, kw = cases[i]
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(300):
                    y = gpu_lib.matvec(*a, **kw)
                torch.cuda.current_stream().synchronize()
            if not torch.equal(y, want[i]):
                errors.append(f"thread {i}: another result")
        except Exception as e:  # noqa: BLE001 (reported below, in the test's own thread)
            errors.append(f"thread {i}: {e}")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_in_a_graph(gpu_lib, fmt, group):
    """16 rows of 6144, captured once and replayed on changing x with eager work between the replays."""
    (x, B, SB, _), kw = _case(fmt, 16, 200, 6144, group, 1)
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn(x.shape, generator=g).to(torch.bfloat16).cuda() for _ in range(3)]
    want = [gpu_lib.matvec(v, B, SB, fmt, **kw) for v in xs]
    y = torch.empty_like(want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.matvec(x, B, SB, fmt, out=y, **kw)
    for i in (1, 0, 2, 1):
        y.zero_()
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
