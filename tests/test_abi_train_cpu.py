"""Host-side refusals of the norm, the grouped bf16 products, the 4-bit
quantiser and product and the gradient clipping: every call here returns
before any device work."""

import ctypes
import os

import pytest
import torch

import moe_grouped_precision_amd as w4a8

P, Q = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
P8 = ctypes.c_void_p((1 << 20) + 8)
P4 = ctypes.c_void_p((1 << 20) + 4)
P2 = ctypes.c_void_p((1 << 20) + 2)
P1 = ctypes.c_void_p((1 << 20) + 1)
NUL = ctypes.c_void_p(0)
NULL, SHAPE, LAYOUT, ALIGN, CAPACITY = 1, 2, 3, 4, 5
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4a8.lib_path()):
        pytest.fail("libw4a8.so is not built (python -m moe_grouped_precision_amd.build)")
    return w4a8.load(require_device=False)


def _caller(f, ok):
    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    return call


def test_rms_norm(lib):
    c = _caller(lib.w4a8_rms_norm, (P, P, P, 1, 4, 256, 1e-6, P, Q, P, P, 0, NUL))
    assert c(a8=P) == SHAPE                                           # y and sum the same buffer
    assert c(a4=-1) == SHAPE and c(a5=0) == SHAPE and c(a5=(1 << 20) + 1) == SHAPE
    assert c(a5=200) == SHAPE                                         # codes need whole groups
    assert c(a6=-1e-9) == SHAPE and c(a6=float("nan")) == SHAPE
    assert c(a3=2) == LAYOUT and c(a11=2) == LAYOUT and c(a11=-1) == LAYOUT
    assert c(a0=NUL) == NULL and c(a9=NUL) == NULL and c(a10=NUL) == NULL
    assert c(a7=NUL, a9=NUL, a10=NUL) == NULL                         # nothing asked for
    assert all(c(**{f"a{i}": P1}) == ALIGN for i in (0, 1, 2, 7, 8))
    assert c(a2=P2, a3=0) == ALIGN and c(a9=P8) == ALIGN and c(a10=P2) == ALIGN
    assert lib.w4a8_last_error() != b""


def test_rms_norm_backward(lib):
    need = lib.w4a8_rms_norm_backward_bytes(4, 256)
    assert need == 4 * 256 * 4 and lib.w4a8_rms_norm_backward_bytes(0, 256) == 0
    assert lib.w4a8_rms_norm_backward_bytes(4, 0) == 0 and lib.w4a8_rms_norm_backward_bytes(-1, 8) == 0
    c = _caller(lib.w4a8_rms_norm_backward, (P, P, 1, P, P, 4, 256, 1e-6, P, P, P, need, NUL))
    assert c(a5=-1) == SHAPE and c(a6=0) == SHAPE and c(a7=-1.0) == SHAPE and c(a2=5) == LAYOUT
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 3, 8, 10))
    assert all(c(**{f"a{i}": P1}) == ALIGN for i in (0, 3, 4, 8)) and c(a9=P2) == ALIGN and c(a10=P2) == ALIGN
    assert c(a11=need - 1) == CAPACITY


@pytest.mark.parametrize("name", ["w4a8_grouped_gemm_bf16", "w4a8_grouped_gemm_dgrad"])
def test_grouped_bf16(lib, name):
    c = _caller(getattr(lib, name), (P, P, P, 16, 4, 64, 32, P, NUL, 0, NUL))
    assert c(a3=-1) == SHAPE and c(a4=0) == SHAPE and c(a4=2049) == SHAPE
    assert c(a5=0) == SHAPE and c(a5=(1 << 24) + 1) == SHAPE and c(a6=0) == SHAPE and c(a6=(1 << 20) + 1) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 1, 2, 7))
    assert all(c(**{f"a{i}": P1}) == ALIGN for i in (0, 1, 7)) and c(a2=P2) == ALIGN


def test_grouped_wgrad(lib):
    c = _caller(lib.w4a8_grouped_gemm_wgrad, (P, P, P, 16, 4, 64, 32, P, 0, 0, NUL, 0, NUL))
    assert c(a3=-1) == SHAPE and c(a4=0) == SHAPE and c(a4=2049) == SHAPE and c(a5=0) == SHAPE and c(a6=0) == SHAPE
    assert c(a8=2) == LAYOUT and c(a8=-1) == LAYOUT
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 1, 2, 7)) and c(a3=0, a7=NUL) == NULL
    assert c(a0=P1) == ALIGN and c(a1=P1) == ALIGN and c(a2=P2) == ALIGN and c(a7=P2) == ALIGN
    assert c(a7=P1, a8=1) == ALIGN


def test_product_workspaces(lib):
    need = lib.w4a8_grouped_gemm_workspace_bytes
    assert need(0, 16, 4, 64, 32) == 0 and need(0, 3, 2, 128, 6000) == 23 * 3 * 128 * 4
    assert need(1, 3, 2, 6000, 128) == 23 * 3 * 128 * 4 and need(2, 8192, 1, 64, 64) == 32 * 64 * 64 * 4
    assert need(3, 3, 2, 128, 8192) == 8 * 3 * 128 * 4
    assert need(4, 3, 2, 128, 6000) == 0 and need(-1, 3, 2, 128, 6000) == 0 and need(0, 0, 2, 128, 6000) == 0
    for f, a in ((lib.w4a8_grouped_gemm_bf16, (P, P, P, 3, 2, 128, 6000, P)),
                 (lib.w4a8_grouped_gemm_dgrad, (P, P, P, 3, 2, 6000, 128, P)),
                 (lib.w4a8_grouped_gemm_wgrad, (P, P, P, 8192, 1, 64, 64, P, 0, 0)),
                 (lib.w4a8_grouped_gemm_a4, (P, P, P, P, P, 3, 2, 128, 8192, P))):
        assert f(*a, Q, 64, NUL) == CAPACITY
        assert f(*a, P8, 1 << 30, NUL) == ALIGN


def test_quantize_fp4(lib):
    need = lib.w4a8_quantize_fp4_bytes(1, 2, 8, 64)
    assert need > 0 and lib.w4a8_quantize_fp4_bytes(0, 2, 8, 64) == 0 and lib.w4a8_quantize_fp4_bytes(1, 0, 8, 64) == 0
    c = _caller(lib.w4a8_quantize_fp4, (P, 1, 2, 8, 64, P, P, P, P, need, NUL))
    assert c(a1=2) == LAYOUT and c(a1=-1) == LAYOUT and c(a1=0) == LAYOUT          # MX has no expert scales
    assert c(a2=0) == SHAPE and c(a2=65537) == SHAPE and c(a3=-1) == SHAPE
    assert c(a4=16) == SHAPE and c(a4=48) == SHAPE and c(a4=0) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 5, 6, 7, 8))
    assert c(a0=P8) == ALIGN and c(a5=P8) == ALIGN and c(a7=P2) == ALIGN and c(a8=P2) == ALIGN
    assert c(a9=need - 1) == CAPACITY


def test_dequantize_fp4(lib):
    c = _caller(lib.w4a8_dequantize_fp4, (P, P, 0, P, 2, 8, 64, P, NUL))
    assert c(a2=2) == LAYOUT and c(a4=0) == SHAPE and c(a5=-1) == SHAPE and c(a6=40) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 1, 7))
    assert c(a0=P8) == ALIGN and c(a3=P2) == ALIGN and c(a7=P8) == ALIGN


def test_quantize_gather_fp4(lib):
    c = _caller(lib.w4a8_quantize_gather_fp4, (P, 4, 64, P, 2, 8, P, P, NUL))
    assert c(a1=-1) == SHAPE and c(a2=48) == SHAPE and c(a2=0) == SHAPE and c(a2=(1 << 20) + 32) == SHAPE
    assert c(a4=0) == SHAPE and c(a5=-1) == SHAPE and c(a1=1 << 30) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 3, 6, 7))
    assert c(a0=P8) == ALIGN and c(a6=P8) == ALIGN and c(a3=P2) == ALIGN


def test_grouped_a4(lib):
    c = _caller(lib.w4a8_grouped_gemm_a4, (P, P, P, P, P, 16, 4, 64, 128, P, NUL, 0, NUL))
    assert c(a5=-1) == SHAPE and c(a6=0) == SHAPE and c(a6=2049) == SHAPE and c(a7=48) == SHAPE and c(a8=64) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 1, 2, 3, 4, 9))
    assert all(c(**{f"a{i}": P8}) == ALIGN for i in (0, 2, 9)) and all(c(**{f"a{i}": P2}) == ALIGN for i in (1, 3, 4))


def _lists(ptrs, numel, types):
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int * n)(*types)


def test_clip_grads(lib):
    a = 1 << 20
    ins, numel, types = _lists([a, a + 4096], [100, 7], [0, 1])
    need = lib.w4a8_clip_grads_bytes(numel, 2)
    assert need == 3 * 8 and lib.w4a8_clip_grads_bytes(numel, -1) == 0
    c = _caller(lib.w4a8_clip_grads, (ins, ins, numel, types, 2, 1.0, 1e-6, P, need, P, NUL))
    assert c(a4=-1) == SHAPE and c(a4=65537) == SHAPE
    assert c(a5=-1.0) == SHAPE and c(a5=float("nan")) == SHAPE and c(a6=-1e-6) == SHAPE and c(a6=float("nan")) == SHAPE
    assert c(a0=NUL) == NULL and c(a2=NUL) == NULL and c(a3=NUL) == NULL and c(a7=NUL) == NULL and c(a9=NUL) == NULL
    assert c(a7=P4) == ALIGN and c(a9=P2) == ALIGN and c(a8=need - 1) == CAPACITY
    assert c(a2=_lists([0], [-1], [0])[1], a4=1) == SHAPE and c(a2=_lists([0], [1 << 44], [0])[1], a4=1) == SHAPE
    assert c(a3=_lists([0, 0], [0, 0], [0, 2])[2]) == LAYOUT
    assert c(a0=_lists([a, 0], [0, 0], [0, 0])[0]) == NULL
    assert c(a0=_lists([a + 2, a + 4096], [0, 0], [0, 0])[0]) == ALIGN
    assert c(a1=_lists([a, a + 4097], [0, 0], [0, 0])[0]) == ALIGN


@pytest.mark.parametrize("ins,outs", [
    ((0, 200), (0, 200)),              # the second tensor starts inside the first
    ((0, 0), (4096, 4396)),            # outputs overlap
    ((0, 1000), (1000, 4096)),         # an output is another tensor
    ((0, 1000), (0, 1004)),            # an output shifted against its tensor
    ((0, 0), (0, 4096)),               # a tensor twice, once in place
])
def test_clip_refuses_overlap(lib, ins, outs):
    a = 1 << 20
    i, numel, types = _lists([a + v for v in ins], [100, 100], [0, 0])
    o = _lists([a + v for v in outs], [0, 0], [0, 0])[0]
    assert lib.w4a8_clip_grads(i, o, numel, types, 2, 1.0, 1e-6, P, BIG, P, NUL) == SHAPE
    assert b"overlap" in lib.w4a8_last_error()


def test_python_refusals_without_a_device():
    t = torch.zeros((2, 64), dtype=torch.bfloat16)
    if torch.cuda.is_available():
        pytest.skip("CPU-only check")
    for call in (lambda: w4a8.rms_norm(t), lambda: w4a8.clip_grads([t], 1.0), lambda: w4a8.quantize_fp4(t, 0)):
        with pytest.raises(RuntimeError, match="MI355X"):
            call()
