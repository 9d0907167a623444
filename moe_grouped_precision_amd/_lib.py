"""ctypes binding of libw4a8.so (argument marshalling only)."""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libw4a8.so")

SCALE_ROW_MAJOR = 0
SCALE_M_MAJOR = 1

_STATUS = {0: "W4A8_OK", 1: "W4A8_ERR_NULL", 2: "W4A8_ERR_SHAPE", 3: "W4A8_ERR_LAYOUT",
           4: "W4A8_ERR_ALIGN", 5: "W4A8_ERR_CAPACITY", 6: "W4A8_ERR_DEVICE", 7: "W4A8_ERR_HIP"}

_lib = None
_ready = set()  # devices that were found to be gfx950
_Tensor, _bfloat16 = torch.Tensor, torch.bfloat16
# without torch.cuda's checks around it: asked only once a device is in _ready
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class W4A8Error(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {detail}")


def lib_path() -> str:
    return _LIB_PATH


def _declare(lib):
    i32, i64, sz, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    lib.w4a8_route_prep.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
    lib.w4a8_route_prep.restype = i32
    lib.w4a8_route_prep_waves.argtypes = [i32, sz]
    lib.w4a8_route_prep_waves.restype = i32
    lib.w4a8_plan_bytes.argtypes = [i32, i64]
    lib.w4a8_plan_bytes.restype = sz
    lib.w4a8_plan.argtypes = [vp, i32, i32, i32, vp, sz, vp]
    lib.w4a8_plan.restype = i32
    lib.w4a8_grouped_gemm.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, vp]
    lib.w4a8_grouped_gemm.restype = i32
    lib.w4a8_grouped_gemm_planned.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, sz, vp, vp]
    lib.w4a8_grouped_gemm_planned.restype = i32
    lib.w4a8_grouped_gemm_planned_noalloc.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, i64, vp, vp]
    lib.w4a8_grouped_gemm_planned_noalloc.restype = i32
    lib.w4a8_grouped_gemm_swiglu.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp]
    lib.w4a8_grouped_gemm_swiglu.restype = i32
    lib.w4a8_grouped_gemm_a16.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, i32, vp, vp]
    lib.w4a8_grouped_gemm_a16.restype = i32
    lib.w4a8_swiglu_quant.argtypes = [vp, i32, i32, vp, vp, i32, vp]
    lib.w4a8_swiglu_quant.restype = i32
    lib.w4a8_combine.argtypes = [vp, i32, i32, vp, vp, i32, i32, vp, vp]
    lib.w4a8_combine.restype = i32
    lib.w4a8_quantize_gather.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, i32, vp]
    lib.w4a8_quantize_gather.restype = i32
    f32 = ctypes.c_float
    lib.w4a8_topk_gate.argtypes = [vp, i32, i32, i32, i32, i32, i32, f32, vp, vp, vp]
    lib.w4a8_topk_gate.restype = i32
    lib.w4a8_topk_gate_backward.argtypes = [vp, i32, i32, i32, vp, vp, i32, i32, i32, f32, vp, vp]
    lib.w4a8_topk_gate_backward.restype = i32
    lib.w4a8_dispatch.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp]
    lib.w4a8_dispatch.restype = i32
    lib.w4a8_dispatch_backward.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp]
    lib.w4a8_dispatch_backward.restype = i32
    lib.w4a8_combine_backward.argtypes = [vp, vp, i32, i32, vp, vp, i32, i32, vp, vp, vp]
    lib.w4a8_combine_backward.restype = i32
    lib.w4a8_matvec.argtypes = [vp, i32, vp, vp, i32, i32, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.w4a8_matvec.restype = i32
    lib.w4a8_swiglu.argtypes = [vp, i32, i32, vp, vp, vp, vp]
    lib.w4a8_swiglu.restype = i32
    lib.w4a8_swiglu_backward.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp]
    lib.w4a8_swiglu_backward.restype = i32
    lib.w4a8_plan_params.argtypes = [ctypes.POINTER(ctypes.c_int32), i32]
    lib.w4a8_plan_params.restype = i32
    lib.w4a8_status_string.argtypes = [i32]
    lib.w4a8_status_string.restype = ctypes.c_char_p
    lib.w4a8_last_error.argtypes = []
    lib.w4a8_last_error.restype = ctypes.c_char_p


def load(require_device: bool = True):
    """Load libw4a8.so (once).  Raises if it is missing, or -- when
    ``require_device`` -- if the current CUDA device is not gfx950."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m moe_grouped_precision_amd.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        _declare(lib)
        _lib = lib
    if require_device and not (_ready and _current_device() in _ready):
        if not torch.cuda.is_available():
            raise RuntimeError("libw4a8 needs a visible MI355X (gfx950) GPU")
        dev = torch.cuda.current_device()
        arch = torch.cuda.get_device_properties(dev).gcnArchName
        if not arch.startswith("gfx950"):
            raise RuntimeError(f"libw4a8 supports gfx950 only, current device is {arch}")
        _ready.add(dev)
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise W4A8Error(fn, status, _lib.w4a8_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# the current stream's handle without a Stream object around it (0.1 against
# 2.7 us, a quarter of a small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_current_device())


def _need(t: torch.Tensor, name: str, dtype, numel: Optional[int] = None):
    if isinstance(t, _Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous() and (
            numel is None or t.numel() == numel):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def plan_params():
    """(GRAN, S_MAX, T_MAX, TN_STREAM, TN_MFMA, header words, tile words)."""
    lib = load(require_device=False)
    out = (ctypes.c_int32 * 7)()
    n = lib.w4a8_plan_params(out, 7)
    return tuple(out[i] for i in range(n))


def plan_bytes(E: int, max_total_rows: int) -> int:
    return int(load(require_device=False).w4a8_plan_bytes(E, max_total_rows))


def route_prep_waves(E: int, lds_limit_bytes: int) -> int:
    """Waves per workgroup the route prep uses for E experts under an LDS limit (0: none fits)."""
    return int(load(require_device=False).w4a8_route_prep_waves(E, lds_limit_bytes))


def route_prep(topk_ids: torch.Tensor, E: int, counts=None, offsets=None, row_of_slot=None):
    """topk_ids int32 [T, top_k] -> (counts [E], expert_offsets [E+1], row_of_slot [T*top_k])."""
    lib = load()
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [T, top_k]")
    T, k = topk_ids.shape
    _need(topk_ids, "topk_ids", torch.int32)
    dev = topk_ids.device
    if counts is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
    if offsets is None:
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    if row_of_slot is None:
        row_of_slot = torch.empty(T * k, dtype=torch.int32, device=dev)
    _need(counts, "counts", torch.int32, E)
    _need(offsets, "expert_offsets", torch.int32, E + 1)
    _need(row_of_slot, "row_of_slot", torch.int32, T * k)
    _check("w4a8_route_prep", lib.w4a8_route_prep(_ptr(topk_ids), T, k, E, _ptr(counts),
                                                 _ptr(offsets), _ptr(row_of_slot), _stream()))
    return counts, offsets, row_of_slot


def plan(expert_offsets: torch.Tensor, E: int, N: int, K: int, max_total_rows: Optional[int] = None,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Device tile plan as an int32 tensor (8-word header + 4 words per m-tile)."""
    lib = load()
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    if out is None:
        if max_total_rows is None:
            raise ValueError("give max_total_rows (an upper bound on offsets[E]) or out")
        nbytes = lib.w4a8_plan_bytes(E, max_total_rows)
        if nbytes == 0:
            raise ValueError("invalid E or max_total_rows")
        out = torch.zeros(nbytes // 4, dtype=torch.int32, device=expert_offsets.device)
    _need(out, "plan", torch.int32)
    _check("w4a8_plan", lib.w4a8_plan(_ptr(expert_offsets), E, N, K, _ptr(out), out.numel() * 4,
                                      _stream()))
    return out


def grouped_gemm(A: torch.Tensor, SA: torch.Tensor, layout: int, B: torch.Tensor, SB: torch.Tensor,
                 expert_offsets: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C[R, N] (torch.bfloat16) of the grouped W4A8 GEMM.

    A uint8 [R, K] E4M3 codes; SA fp32 [R, K/128] (layout 0) or [K/128, R]
    (layout 1); B uint8 [E, N, K/2] packed E2M1; SB uint8 [E, N, K/32] E8M0;
    expert_offsets int32 [E+1] with offsets[E] == R.
    """
    lib = load()
    if A.dim() != 2 or B.dim() != 3 or SB.dim() != 3:
        raise ValueError("A must be [R, K], B [E, N, K/2], SB [E, N, K/32]")
    R, K = A.shape
    E, N, Kh = B.shape
    if Kh * 2 != K or SB.shape != (E, N, K // 32):
        raise ValueError("inconsistent K between A, B and SB")
    _need(A, "A", torch.uint8)
    _need(SA, "a_scales", torch.float32, R * (K // 128))
    _need(B, "B", torch.uint8)
    _need(SB, "b_scales", torch.uint8)
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=A.device)
    if out.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("out must be bfloat16 (or 16-bit integer bits)")
    _need(out, "out", out.dtype, R * N)
    if R == 0:
        return out  # no rows: nothing to compute
    _check("w4a8_grouped_gemm", lib.w4a8_grouped_gemm(
        _ptr(A), _ptr(SA), int(layout), _ptr(B), _ptr(SB), _ptr(expert_offsets), E, N, K,
        _ptr(out), _stream()))
    return out


WSCALE_MX = 0  # MXFP4 weight scales: E8M0 per 32 K
WSCALE_NV = 1  # NVFP4 weight scales: E4M3 per 16 K


def grouped_gemm_a16(A: torch.Tensor, B: torch.Tensor, SB: torch.Tensor, fmt: int, expert_offsets: torch.Tensor,
                     expert_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C[R, N] (bf16) of the grouped GEMM with bf16 activations and FP4
    weights.  A bf16 (or 16-bit integer bits) [R, K]; B uint8 [E, N, K/2]
    packed E2M1; SB uint8 [E, N, K/32] E8M0 (fmt WSCALE_MX) or [E, N, K/16]
    E4M3 (fmt WSCALE_NV); expert_scales fp32 [E] or None; expert_offsets
    int32 [E+1] with offsets[E] == R."""
    lib = load()
    if A.dim() != 2 or B.dim() != 3 or SB.dim() != 3:
        raise ValueError("A must be [R, K], B [E, N, K/2], SB [E, N, K/blk]")
    R, K = A.shape
    E, N, Kh = B.shape
    blk = 32 if fmt == WSCALE_MX else 16
    if Kh * 2 != K or SB.shape != (E, N, K // blk):
        raise ValueError("inconsistent K between A, B and SB")
    if A.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("A must be bfloat16 (or 16-bit integer bits)")
    _need(A, "A", A.dtype)
    _need(B, "B", torch.uint8)
    _need(SB, "b_scales", torch.uint8)
    if expert_scales is not None:
        _need(expert_scales, "expert_scales", torch.float32, E)
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=A.device)
    if out.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("out must be bfloat16 (or 16-bit integer bits)")
    _need(out, "out", out.dtype, R * N)
    if R == 0:
        return out
    _check("w4a8_grouped_gemm_a16", lib.w4a8_grouped_gemm_a16(
        _ptr(A), _ptr(B), _ptr(SB), int(fmt), _ptr(expert_scales), _ptr(expert_offsets), E, N, K,
        _ptr(out), _stream()))
    return out


def grouped_gemm_planned(A: torch.Tensor, SA: torch.Tensor, layout: int, B: torch.Tensor, SB: torch.Tensor,
                         expert_offsets: torch.Tensor, plan: torch.Tensor,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C[R, N] (bf16) of the grouped W4A8 GEMM over a tile list `plan` (int32,
    w4a8_plan's format, e.g. the output of plan()); the rest as grouped_gemm."""
    lib = load()
    if A.dim() != 2 or B.dim() != 3 or SB.dim() != 3:
        raise ValueError("A must be [R, K], B [E, N, K/2], SB [E, N, K/32]")
    R, K = A.shape
    E, N, Kh = B.shape
    if Kh * 2 != K or SB.shape != (E, N, K // 32):
        raise ValueError("inconsistent K between A, B and SB")
    _need(A, "A", torch.uint8)
    _need(SA, "a_scales", torch.float32, R * (K // 128))
    _need(B, "B", torch.uint8)
    _need(SB, "b_scales", torch.uint8)
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    _need(plan, "plan", torch.int32)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=A.device)
    if out.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("out must be bfloat16 (or 16-bit integer bits)")
    _need(out, "out", out.dtype, R * N)
    if R == 0:
        return out
    _check("w4a8_grouped_gemm_planned", lib.w4a8_grouped_gemm_planned(
        _ptr(A), _ptr(SA), int(layout), _ptr(B), _ptr(SB), _ptr(expert_offsets), E, N, K, _ptr(plan),
        plan.numel() * 4, _ptr(out), _stream()))
    return out


def grouped_gemm_planned_noalloc(A: torch.Tensor, SA: torch.Tensor, layout: int, B: torch.Tensor,
                                 SB: torch.Tensor, expert_offsets: torch.Tensor, out: torch.Tensor,
                                 max_total_rows: Optional[int] = None) -> torch.Tensor:
    """The planned GEMM with its plan in the library's device scratch: nothing
    is allocated, so `out` (bf16 [R, N]) must be given; max_total_rows
    defaults to R = A.shape[0]."""
    lib = load()
    if A.dim() != 2 or B.dim() != 3 or SB.dim() != 3:
        raise ValueError("A must be [R, K], B [E, N, K/2], SB [E, N, K/32]")
    R, K = A.shape
    E, N, Kh = B.shape
    if Kh * 2 != K or SB.shape != (E, N, K // 32):
        raise ValueError("inconsistent K between A, B and SB")
    _need(A, "A", torch.uint8)
    _need(SA, "a_scales", torch.float32, R * (K // 128))
    _need(B, "B", torch.uint8)
    _need(SB, "b_scales", torch.uint8)
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    if out.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("out must be bfloat16 (or 16-bit integer bits)")
    _need(out, "out", out.dtype, R * N)
    if R == 0:
        return out
    _check("w4a8_grouped_gemm_planned_noalloc", lib.w4a8_grouped_gemm_planned_noalloc(
        _ptr(A), _ptr(SA), int(layout), _ptr(B), _ptr(SB), _ptr(expert_offsets), E, N, K,
        int(R if max_total_rows is None else max_total_rows), _ptr(out), _stream()))
    return out


def grouped_gemm_swiglu(A: torch.Tensor, SA: torch.Tensor, layout: int, B13: torch.Tensor, SB13: torch.Tensor,
                        expert_offsets: torch.Tensor, layout2: int, A2: Optional[torch.Tensor] = None,
                        SA2: Optional[torch.Tensor] = None):
    """The gate/up GEMM with SwiGLU and E4M3 requantization in its epilogue:
    (A2 uint8 [R, I] codes of silu(gate) * up, SA2 fp32 [R, I/128] for layout2
    0 or [I/128, R] for layout2 1).  B13 uint8 [E, 2I, K/2] (gate columns
    first), SB13 uint8 [E, 2I, K/32]; the rest as grouped_gemm."""
    lib = load()
    if A.dim() != 2 or B13.dim() != 3 or SB13.dim() != 3:
        raise ValueError("A must be [R, K], B13 [E, 2I, K/2], SB13 [E, 2I, K/32]")
    R, K = A.shape
    E, N2, Kh = B13.shape
    if Kh * 2 != K or N2 % 2 or SB13.shape != (E, N2, K // 32):
        raise ValueError("inconsistent shapes between A, B13 and SB13")
    I = N2 // 2
    _need(A, "A", torch.uint8)
    _need(SA, "a_scales", torch.float32, R * (K // 128))
    _need(B13, "B13", torch.uint8)
    _need(SB13, "b13_scales", torch.uint8)
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    if A2 is None:
        A2 = torch.empty((R, I), dtype=torch.uint8, device=A.device)
    if SA2 is None:
        SA2 = torch.empty((R, I // 128) if layout2 == 0 else (I // 128, R), dtype=torch.float32, device=A.device)
    _need(A2, "A2", torch.uint8, R * I)
    _need(SA2, "a2_scales", torch.float32, R * (I // 128))
    if R == 0:
        return A2, SA2
    _check("w4a8_grouped_gemm_swiglu", lib.w4a8_grouped_gemm_swiglu(
        _ptr(A), _ptr(SA), int(layout), _ptr(B13), _ptr(SB13), _ptr(expert_offsets), E, I, K, _ptr(A2),
        _ptr(SA2), int(layout2), _stream()))
    return A2, SA2


def quantize_gather(x: torch.Tensor, row_of_slot: torch.Tensor, top_k: int, R: int, layout: int,
                    A: Optional[torch.Tensor] = None, SA: Optional[torch.Tensor] = None):
    """bf16 tokens x [T, K] -> (A uint8 [R, K] E4M3 codes, SA fp32 scales) written
    to the grouped row of every slot (row_of_slot int32 [T * top_k]); SA is
    [R, K/128] for layout 0 and [K/128, R] for layout 1."""
    lib = load()
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    T, K = x.shape
    if x.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("x must be bfloat16 (or 16-bit integer bits)")
    _need(x, "x", x.dtype)
    _need(row_of_slot, "row_of_slot", torch.int32, T * top_k)
    if A is None:
        A = torch.zeros((R, K), dtype=torch.uint8, device=x.device)
    if SA is None:
        shape = (R, K // 128) if layout == 0 else (K // 128, R)
        SA = torch.zeros(shape, dtype=torch.float32, device=x.device)
    _need(A, "A", torch.uint8, R * K)
    _need(SA, "a_scales", torch.float32, R * (K // 128))
    _check("w4a8_quantize_gather", lib.w4a8_quantize_gather(
        _ptr(x), T, K, _ptr(row_of_slot), int(top_k), int(R), _ptr(A), _ptr(SA), int(layout), _stream()))
    return A, SA


def combine(C: torch.Tensor, row_of_slot: torch.Tensor, weights: torch.Tensor, top_k: int,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t, :] (bf16) = sum_j weights[t*top_k + j] * C[row_of_slot[t*top_k + j], :],
    fp32 in slot order; C [R, N] bf16 grouped rows, row_of_slot int32 and
    weights fp32 of T*top_k slots."""
    lib = load()
    if C.dim() != 2:
        raise ValueError("C must be [R, N]")
    R, N = C.shape
    if C.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("C must be bfloat16 (or 16-bit integer bits)")
    _need(C, "C", C.dtype)
    if row_of_slot.numel() % top_k:
        raise ValueError("row_of_slot must hold T * top_k entries")
    T = row_of_slot.numel() // top_k
    _need(row_of_slot, "row_of_slot", torch.int32, T * top_k)
    _need(weights, "weights", torch.float32, T * top_k)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=C.device)
    if out.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("out must be bfloat16 (or 16-bit integer bits)")
    _need(out, "out", out.dtype, T * N)
    _check("w4a8_combine", lib.w4a8_combine(_ptr(C), R, N, _ptr(row_of_slot), _ptr(weights), T, int(top_k),
                                            _ptr(out), _stream()))
    return out


def swiglu_quant(C: torch.Tensor, layout: int, A: Optional[torch.Tensor] = None, SA: Optional[torch.Tensor] = None):
    """Gate/up output C [R, 2I] (bf16; gate columns first) -> (A uint8 [R, I]
    E4M3 codes of silu(gate) * up, SA fp32 scales [R, I/128] for layout 0 or
    [I/128, R] for layout 1)."""
    lib = load()
    if C.dim() != 2 or C.shape[1] % 2:
        raise ValueError("C must be [R, 2I]")
    R, I = C.shape[0], C.shape[1] // 2
    if C.dtype not in (torch.bfloat16, torch.uint16, torch.int16):
        raise TypeError("C must be bfloat16 (or 16-bit integer bits)")
    _need(C, "C", C.dtype)
    if A is None:
        A = torch.empty((R, I), dtype=torch.uint8, device=C.device)
    if SA is None:
        SA = torch.empty((R, I // 128) if layout == 0 else (I // 128, R), dtype=torch.float32, device=C.device)
    _need(A, "A", torch.uint8, R * I)
    _need(SA, "a_scales", torch.float32, R * (I // 128))
    _check("w4a8_swiglu_quant", lib.w4a8_swiglu_quant(_ptr(C), R, I, _ptr(A), _ptr(SA), int(layout), _stream()))
    return A, SA


GATE_SOFTMAX = 0
GATE_SIGMOID = 1


def _logits_type(t: torch.Tensor) -> int:
    if t.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")
    return 0 if t.dtype == torch.float32 else 1


def _bf16(t: torch.Tensor, name: str, numel: Optional[int] = None):
    dtype = getattr(t, "dtype", None)
    if dtype is not _bfloat16 and isinstance(t, _Tensor) and dtype not in (torch.uint16, torch.int16):
        raise TypeError(f"{name} must be bfloat16 (or 16-bit integer bits)")
    _need(t, name, dtype, numel)


def topk_gate(logits: torch.Tensor, top_k: int, score: int = GATE_SOFTMAX, renorm: bool = True, scale: float = 1.0,
              ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None):
    """Router logits [T, E] (fp32 or bf16) -> (ids int32 [T, top_k] by
    descending logit, ties to the lower expert; weights fp32 [T, top_k]).
    Weights are scale times the softmax over all experts or the sigmoid, with
    renorm divided by their sum over the selected; -inf closes an expert, and
    a slot with nothing left is id -1, weight 0."""
    lib = load()
    kind = _logits_type(logits)
    T, E = logits.shape
    _need(logits, "logits", logits.dtype)
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    _need(ids, "ids", torch.int32, T * top_k)
    _need(weights, "weights", torch.float32, T * top_k)
    _check("w4a8_topk_gate", lib.w4a8_topk_gate(_ptr(logits), kind, T, E, int(top_k), int(score), int(renorm),
                                                float(scale), _ptr(ids), _ptr(weights), _stream()))
    return ids, weights


def topk_gate_backward(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, score: int = GATE_SOFTMAX,
                       renorm: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dlogits [T, E] (the logits' type) from dweights fp32 [T, top_k]; logits,
    score, renorm and scale as given to topk_gate, ids as it returned them.
    out must not be the logits."""
    lib = load()
    kind = _logits_type(logits)
    T, E = logits.shape
    _need(logits, "logits", logits.dtype)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError("ids must be [T, top_k]")
    k = ids.shape[1]
    _need(ids, "ids", torch.int32)
    _need(dweights, "dweights", torch.float32, T * k)
    if out is None:
        out = torch.empty_like(logits)
    _need(out, "out", logits.dtype, T * E)
    _check("w4a8_topk_gate_backward", lib.w4a8_topk_gate_backward(
        _ptr(logits), kind, T, E, _ptr(ids), _ptr(dweights), k, int(score), int(renorm), float(scale), _ptr(out),
        _stream()))
    return out


def _slots(row_of_slot: torch.Tensor, top_k: int) -> int:
    if top_k < 1 or row_of_slot.numel() % top_k:
        raise ValueError("row_of_slot must hold T * top_k entries")
    _need(row_of_slot, "row_of_slot", torch.int32)
    return row_of_slot.numel() // top_k


def dispatch(x: torch.Tensor, row_of_slot: torch.Tensor, top_k: int, R: int,
             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 tokens x [T, K] -> A bf16 [R, K], every token copied to the rows of
    its slots (row_of_slot int32 [T * top_k]; slots without a row are skipped,
    rows without a slot keep what `out` holds, zeros where it is not given)."""
    lib = load()
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    T, K = x.shape
    _bf16(x, "x")
    _need(row_of_slot, "row_of_slot", torch.int32, T * top_k)
    if out is None:
        out = torch.zeros((R, K), dtype=torch.bfloat16, device=x.device)
    _bf16(out, "out", R * K)
    _check("w4a8_dispatch", lib.w4a8_dispatch(_ptr(x), T, K, _ptr(row_of_slot), int(top_k), int(R), _ptr(out),
                                              _stream()))
    return out


def dispatch_backward(dA: torch.Tensor, row_of_slot: torch.Tensor, top_k: int,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx bf16 [T, K] of dispatch: every token's sum of its slots' rows of dA
    bf16 [R, K], in fp32, rounded once."""
    lib = load()
    if dA.dim() != 2:
        raise ValueError("dA must be [R, K]")
    R, K = dA.shape
    _bf16(dA, "dA")
    T = _slots(row_of_slot, top_k)
    if out is None:
        out = torch.empty((T, K), dtype=torch.bfloat16, device=dA.device)
    _bf16(out, "out", T * K)
    _check("w4a8_dispatch_backward", lib.w4a8_dispatch_backward(_ptr(dA), R, K, _ptr(row_of_slot), T, int(top_k),
                                                                _ptr(out), _stream()))
    return out


def combine_backward(C: torch.Tensor, dout: torch.Tensor, row_of_slot: torch.Tensor, weights: torch.Tensor,
                     top_k: int, dC: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None):
    """Gradients of combine: (dC bf16 [R, N] = weight * dout in the row of each
    slot, dweights fp32 [T * top_k] = <C row, dout row>, 0 for slots without a
    row).  Rows of dC without a slot keep what dC holds, zeros where it is not
    given."""
    lib = load()
    if C.dim() != 2 or dout.dim() != 2 or dout.shape[1] != C.shape[1]:
        raise ValueError("C must be [R, N] and dout [T, N]")
    R, N = C.shape
    T = _slots(row_of_slot, top_k)
    _bf16(C, "C")
    _bf16(dout, "dout", T * N)
    _need(weights, "weights", torch.float32, T * top_k)
    if dC is None:
        dC = torch.zeros((R, N), dtype=torch.bfloat16, device=C.device)
    if dweights is None:
        dweights = torch.empty(T * top_k, dtype=torch.float32, device=C.device)
    _bf16(dC, "dC", R * N)
    _need(dweights, "dweights", torch.float32, T * top_k)
    _check("w4a8_combine_backward", lib.w4a8_combine_backward(
        _ptr(C), _ptr(dout), R, N, _ptr(row_of_slot), _ptr(weights), T, int(top_k), _ptr(dC), _ptr(dweights),
        _stream()))
    return dC, dweights


WSCALE_INT4 = 2  # integer codes 0..15, bf16 scale per 32, 64 or 128 K (matvec)


def matvec(x: torch.Tensor, B: torch.Tensor, SB: torch.Tensor, fmt: int, expert_ids: Optional[torch.Tensor] = None,
           expert_scales: Optional[torch.Tensor] = None, zeros: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[S, N] (bf16) of a few tokens with 4-bit weights: slot s multiplies row
    s // (S / X) of x bf16 [X, K] with the weights of expert expert_ids[s]
    (int32, S = their number, at most 64; an id outside [0, E) gives zeros;
    None: one weight matrix, S = X).  B uint8 [E, N, K/2]; SB uint8 [E, N,
    K/32] E8M0 (fmt WSCALE_MX), uint8 [E, N, K/16] E4M3 (WSCALE_NV) or bf16
    [E, N, K/group] (WSCALE_INT4) with optional zeros uint8 of the same shape
    (8 where not given); expert_scales fp32 [E] or None."""
    lib = load()
    if x.dim() != 2 or B.dim() != 3 or SB.dim() != 3:
        raise ValueError("x must be [X, K], B [E, N, K/2], SB [E, N, K/group]")
    X, K = x.shape
    E, N, Kh = B.shape
    if Kh * 2 != K or SB.shape[:2] != B.shape[:2]:
        raise ValueError("inconsistent shapes of x, B and SB")
    groups = SB.shape[2]
    if groups < 1 or K % groups:
        raise ValueError("SB must hold a whole number of groups of K")
    _bf16(x, "x")
    _need(B, "B", torch.uint8)
    _need(SB, "b_scales", torch.bfloat16 if fmt == WSCALE_INT4 else torch.uint8)
    if zeros is not None:
        _need(zeros, "zeros", torch.uint8, E * N * groups)
    if expert_scales is not None:
        _need(expert_scales, "expert_scales", torch.float32, E)
    S = X
    if expert_ids is not None:
        _need(expert_ids, "expert_ids", torch.int32)
        S = expert_ids.numel()
    if out is None:
        out = torch.empty((S, N), dtype=torch.bfloat16, device=x.device)
    _bf16(out, "out", S * N)
    _check("w4a8_matvec", lib.w4a8_matvec(
        _ptr(x), X, _ptr(B), _ptr(SB), int(fmt), K // groups, _ptr(zeros), _ptr(expert_scales), _ptr(expert_ids), S, E,
        N, K, _ptr(out), _stream()))
    return out


def swiglu(C: torch.Tensor, checkpoint: bool = False, h: Optional[torch.Tensor] = None,
           codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """Gate/up output C bf16 [R, 2I] (gate columns first) -> h bf16 [R, I] =
    silu(gate) * up; with checkpoint, (h, codes uint8 [R, 2I], scales fp32
    [R, 2I/128]): an E4M3 copy of C for swiglu_backward."""
    lib = load()
    if C.dim() != 2 or C.shape[1] % 2:
        raise ValueError("C must be [R, 2I]")
    R, I = C.shape[0], C.shape[1] // 2
    _bf16(C, "C")
    if not checkpoint and (codes is not None or scales is not None):
        raise ValueError("codes and scales go with checkpoint=True")
    if h is None:
        h = torch.empty((R, I), dtype=torch.bfloat16, device=C.device)
    _bf16(h, "h", R * I)
    if checkpoint:
        if codes is None:
            codes = torch.empty((R, 2 * I), dtype=torch.uint8, device=C.device)
        if scales is None:
            scales = torch.empty((R, 2 * I // 128), dtype=torch.float32, device=C.device)
        _need(codes, "codes", torch.uint8, R * 2 * I)
        _need(scales, "scales", torch.float32, R * (2 * I // 128))
    _check("w4a8_swiglu", lib.w4a8_swiglu(_ptr(C), R, I, _ptr(h), _ptr(codes), _ptr(scales), _stream()))
    return (h, codes, scales) if checkpoint else h


def swiglu_backward(codes: torch.Tensor, scales: torch.Tensor, dh: torch.Tensor, dC: Optional[torch.Tensor] = None,
                    h: Optional[torch.Tensor] = None):
    """dC bf16 [R, 2I] of swiglu from its 8-bit copy (codes uint8 [R, 2I],
    scales fp32 [R, 2I/128]) and dh bf16 [R, I].  With h (bf16 [R, I]) given,
    the recomputed h is written there and (dC, h) returned."""
    lib = load()
    if dh.dim() != 2:
        raise ValueError("dh must be [R, I]")
    R, I = dh.shape
    _bf16(dh, "dh")
    _need(codes, "codes", torch.uint8, R * 2 * I)
    _need(scales, "scales", torch.float32, R * (2 * I // 128))
    if dC is None:
        dC = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=dh.device)
    _bf16(dC, "dC", R * 2 * I)
    if h is not None:
        _bf16(h, "h", R * I)
    _check("w4a8_swiglu_backward", lib.w4a8_swiglu_backward(_ptr(codes), _ptr(scales), _ptr(dh), R, I, _ptr(dC),
                                                            _ptr(h), _stream()))
    return dC if h is None else (dC, h)
