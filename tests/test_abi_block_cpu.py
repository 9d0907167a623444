"""Host-side refusals of the operators around the expert products: every call
here returns before any device work."""

import ctypes
import os

import pytest

import moe_grouped_precision_amd as w4a8

P = ctypes.c_void_p(1 << 20)
P8 = ctypes.c_void_p((1 << 20) + 8)
P2 = ctypes.c_void_p((1 << 20) + 2)
P1 = ctypes.c_void_p((1 << 20) + 1)
NUL = ctypes.c_void_p(0)
NULL, SHAPE, LAYOUT, ALIGN = 1, 2, 3, 4


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


def test_topk_gate(lib):
    c = _caller(lib.w4a8_topk_gate, (P, 0, 4, 32, 8, 0, 1, 1.0, P, P, NUL))
    assert c(a2=-1) == SHAPE and c(a3=0) == SHAPE and c(a3=16385) == SHAPE
    assert c(a4=0) == SHAPE and c(a4=33) == SHAPE and c(a3=100, a4=65) == SHAPE
    assert c(a2=1 << 30) == SHAPE                                     # T * top_k
    assert c(a1=2) == LAYOUT and c(a5=2) == LAYOUT and c(a5=-1) == LAYOUT
    assert c(a0=NUL) == NULL and c(a8=NUL) == NULL and c(a9=NUL) == NULL
    assert c(a0=P2) == ALIGN and c(a1=1, a0=P1) == ALIGN and c(a8=P2) == ALIGN and c(a9=P2) == ALIGN
    assert lib.w4a8_last_error() != b""


def test_topk_gate_backward(lib):
    c = _caller(lib.w4a8_topk_gate_backward, (P, 0, 4, 32, P, P, 8, 0, 1, 1.0, P, NUL))
    assert c(a2=-1) == SHAPE and c(a3=16385) == SHAPE and c(a6=0) == SHAPE and c(a6=33) == SHAPE
    assert c(a1=3) == LAYOUT and c(a7=2) == LAYOUT
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 4, 5, 10))
    assert all(c(**{f"a{i}": P2}) == ALIGN for i in (0, 4, 5, 10))


def test_dispatch(lib):
    c = _caller(lib.w4a8_dispatch, (P, 4, 64, P, 2, 8, P, NUL))
    assert c(a1=-1) == SHAPE and c(a2=0) == SHAPE and c(a2=(1 << 24) + 1) == SHAPE
    assert c(a4=0) == SHAPE and c(a5=-1) == SHAPE and c(a1=1 << 30) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 3, 6))
    assert c(a0=P1) == ALIGN and c(a6=P1) == ALIGN and c(a3=P2) == ALIGN


def test_dispatch_backward(lib):
    c = _caller(lib.w4a8_dispatch_backward, (P, 8, 64, P, 4, 2, P, NUL))
    assert c(a1=-1) == SHAPE and c(a2=0) == SHAPE and c(a4=-1) == SHAPE and c(a5=0) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 3, 6))
    assert c(a0=P1) == ALIGN and c(a6=P1) == ALIGN and c(a3=P2) == ALIGN


def test_combine_backward(lib):
    c = _caller(lib.w4a8_combine_backward, (P, P, 8, 64, P, P, 4, 2, P, P, NUL))
    assert c(a2=-1) == SHAPE and c(a3=0) == SHAPE and c(a6=-1) == SHAPE and c(a7=0) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 1, 4, 5, 8, 9))
    assert all(c(**{f"a{i}": P1}) == ALIGN for i in (0, 1, 8)) and all(c(**{f"a{i}": P2}) == ALIGN for i in (4, 5, 9))


def test_matvec(lib):
    c = _caller(lib.w4a8_matvec, (P, 2, P, P, 2, 64, NUL, NUL, P, 4, 8, 48, 512, P, NUL))
    assert c(a4=3) == LAYOUT and c(a4=-1) == LAYOUT
    assert c(a5=16) == SHAPE and c(a5=256) == SHAPE and c(a4=0) == SHAPE and c(a4=1, a5=32) == SHAPE
    assert c(a4=0, a5=32, a6=P) == LAYOUT                             # zero points with MXFP4
    assert c(a9=-1) == SHAPE and c(a9=65, a1=1) == SHAPE and c(a9=5) == SHAPE and c(a1=0) == SHAPE
    assert c(a10=0) == SHAPE and c(a10=65537) == SHAPE and c(a8=NUL) == SHAPE   # E > 1 without ids
    assert c(a11=0) == SHAPE and c(a12=0) == SHAPE and c(a12=544) == SHAPE and c(a12=(1 << 20) + 64) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 2, 3, 13))
    assert c(a0=P8) == ALIGN and c(a2=P8) == ALIGN and all(c(**{f"a{i}": P2}) == ALIGN for i in (3, 6, 7, 8, 13))


def test_swiglu(lib):
    c = _caller(lib.w4a8_swiglu, (P, 8, 256, P, P, P, NUL))
    assert c(a1=-1) == SHAPE and c(a2=200) == SHAPE and c(a2=0) == SHAPE and c(a2=(1 << 20) + 128) == SHAPE
    assert c(a1=(1 << 31) - 1, a2=1 << 20) == SHAPE
    assert c(a0=NUL) == NULL and c(a3=NUL) == NULL and c(a4=NUL) == NULL and c(a5=NUL) == NULL
    assert c(a0=P8) == ALIGN and c(a3=P8) == ALIGN and c(a4=P8) == ALIGN and c(a5=P2) == ALIGN


def test_swiglu_backward(lib):
    c = _caller(lib.w4a8_swiglu_backward, (P, P, P, 8, 256, P, NUL, NUL))
    assert c(a3=-1) == SHAPE and c(a4=200) == SHAPE and c(a3=(1 << 31) - 1, a4=1 << 20) == SHAPE
    assert all(c(**{f"a{i}": NUL}) == NULL for i in (0, 1, 2, 5))
    assert all(c(**{f"a{i}": P8}) == ALIGN for i in (0, 2, 5, 6)) and c(a1=P2) == ALIGN
