"""ctypes binding of libw4a8.so (argument marshalling only)."""

from __future__ import annotations

import ctypes
import os
from array import array
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
    lib.w4a8_rms_norm.argtypes = [vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp, i32, vp]
    lib.w4a8_rms_norm.restype = i32
    lib.w4a8_rms_norm_backward.argtypes = [vp, vp, i32, vp, vp, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.w4a8_rms_norm_backward.restype = i32
    lib.w4a8_rms_norm_backward_bytes.argtypes = [i32, i32]
    lib.w4a8_rms_norm_backward_bytes.restype = sz
    for f in (lib.w4a8_grouped_gemm_bf16, lib.w4a8_grouped_gemm_dgrad):
        f.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]
        f.restype = i32
    lib.w4a8_grouped_gemm_wgrad.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, i32, i32, vp, sz, vp]
    lib.w4a8_grouped_gemm_wgrad.restype = i32
    lib.w4a8_quantize_fp4.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.w4a8_quantize_fp4.restype = i32
    lib.w4a8_quantize_fp4_bytes.argtypes = [i32, i32, i32, i32]
    lib.w4a8_quantize_fp4_bytes.restype = sz
    lib.w4a8_dequantize_fp4.argtypes = [vp, vp, i32, vp, i32, i32, i32, vp, vp]
    lib.w4a8_dequantize_fp4.restype = i32
    lib.w4a8_quantize_gather_fp4.argtypes = [vp, i32, i32, vp, i32, i32, vp, vp, vp]
    lib.w4a8_quantize_gather_fp4.restype = i32
    lib.w4a8_grouped_gemm_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.w4a8_grouped_gemm_workspace_bytes.restype = sz
    lib.w4a8_grouped_gemm_tile.argtypes = [i32, i32, i32, i32, i32]
    lib.w4a8_grouped_gemm_tile.restype = i32
    lib.w4a8_grouped_gemm_a4.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]
    lib.w4a8_grouped_gemm_a4.restype = i32
    lib.w4a8_clip_grads.argtypes = [vp, vp, vp, vp, i32, f32, f32, vp, sz, vp, vp]
    lib.w4a8_clip_grads.restype = i32
    lib.w4a8_clip_grads_bytes.argtypes = [vp, i32]
    lib.w4a8_clip_grads_bytes.restype = sz
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


def _here(*tensors: Optional[torch.Tensor]):
    """The tensors live on the current device, whose stream the call uses."""
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors must be on the current device (cuda:{dev}), got {t.device}")


def _weight_type(w: Optional[torch.Tensor], K: int, name: str = "weight") -> int:
    if w is None:
        return 0
    if isinstance(w, _Tensor) and w.dtype not in (torch.float32, _bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16, got {w.dtype}")
    _need(w, name, getattr(w, "dtype", None), K)
    return 0 if w.dtype is torch.float32 else 1


def _rms_norm(x, weight, eps, residual, y, sum_out, A, SA, layout):
    T, K = x.shape
    kind = _weight_type(weight, K)
    _here(x, weight, residual, y, sum_out, A, SA)
    _check("w4a8_rms_norm", load().w4a8_rms_norm(
        _ptr(x), _ptr(residual), _ptr(weight), kind, T, K, float(eps), _ptr(y), _ptr(sum_out), _ptr(A), _ptr(SA),
        int(layout), _stream()))


def _norm_inputs(x, residual, sum_out):
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    _bf16(x, "x")
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out goes with a residual")
        return None
    _bf16(residual, "residual", x.numel())
    if sum_out is None:
        sum_out = torch.empty(x.shape, dtype=_bfloat16, device=x.device)
    _bf16(sum_out, "sum_out", x.numel())
    return sum_out


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
             sum_out: Optional[torch.Tensor] = None):
    """y bf16 [T, K] = h / sqrt(mean(h^2) + eps) * weight of x bf16 [T, K]; with
    residual bf16 [T, K], (y, h) with h = bf16(x + residual), otherwise h = x.
    weight fp32 or bf16 [K], or None for ones.  out and sum_out may be x or
    residual."""
    load()
    sum_out = _norm_inputs(x, residual, sum_out)
    if out is None:
        out = torch.empty(x.shape, dtype=_bfloat16, device=x.device)
    _bf16(out, "out", x.numel())
    _rms_norm(x, weight, eps, residual, out, sum_out, None, None, 0)
    return out if residual is None else (out, sum_out)


def rms_norm_quant(x: torch.Tensor, weight: Optional[torch.Tensor], layout: int, eps: float = 1e-6,
                   residual: Optional[torch.Tensor] = None, A: Optional[torch.Tensor] = None,
                   SA: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None):
    """The same norm in 8 bits, the input of grouped_gemm: (A uint8 [T, K] E4M3
    codes, SA fp32 [T, K/128] for layout 0 or [K/128, T] for layout 1), with
    residual (A, SA, h).  out bf16 [T, K], where given, gets y too."""
    load()
    sum_out = _norm_inputs(x, residual, sum_out)
    T, K = x.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    if A is None:
        A = torch.empty((T, K), dtype=torch.uint8, device=x.device)
    if SA is None:
        SA = torch.empty((T, K // 128) if layout == 0 else (K // 128, T), dtype=torch.float32, device=x.device)
    _need(A, "A", torch.uint8, T * K)
    _need(SA, "a_scales", torch.float32, T * (K // 128))
    if out is not None:
        _bf16(out, "out", T * K)
    _rms_norm(x, weight, eps, residual, out, sum_out, A, SA, layout)
    return (A, SA) if residual is None else (A, SA, sum_out)


def rms_norm_backward(h: torch.Tensor, weight: Optional[torch.Tensor], dy: torch.Tensor, eps: float = 1e-6,
                      dh: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                      dweight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """(dx bf16 [T, K], dweight fp32 [K]) of rms_norm from h, its sum (its x
    without a residual), and dy bf16 [T, K]; dh bf16 [T, K], the gradient that
    reaches h beside y, is added.  dx is the gradient of x and of residual; it
    may be the buffer of dy, dh or h."""
    lib = load()
    if h.dim() != 2:
        raise ValueError("h must be [T, K]")
    T, K = h.shape
    _bf16(h, "h")
    kind = _weight_type(weight, K)
    _bf16(dy, "dy", T * K)
    if dh is not None:
        _bf16(dh, "dh", T * K)
    if dx is None:
        dx = torch.empty((T, K), dtype=_bfloat16, device=h.device)
    if dweight is None:
        dweight = torch.empty(K, dtype=torch.float32, device=h.device)
    _bf16(dx, "dx", T * K)
    _need(dweight, "dweight", torch.float32, K)
    need = lib.w4a8_rms_norm_backward_bytes(T, K)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=h.device)
    _need(workspace, "workspace", torch.uint8)
    _here(h, weight, dy, dh, dx, dweight, workspace)
    _check("w4a8_rms_norm_backward", lib.w4a8_rms_norm_backward(
        _ptr(h), _ptr(weight), kind, _ptr(dy), _ptr(dh), T, K, float(eps), _ptr(dx), _ptr(dweight), _ptr(workspace),
        workspace.numel(), _stream()))
    return dx, dweight


def _product(rows: torch.Tensor, W: torch.Tensor, expert_offsets: torch.Tensor, axis: int):
    """Shapes of a product of rows with bf16 weights; axis: of W that the rows have."""
    if rows.dim() != 2 or W.dim() != 3:
        raise ValueError("rows must be two-dimensional, W [E, N, K]")
    if rows.shape[1] != W.shape[axis]:
        raise ValueError("inconsistent shapes of the rows and W")
    _need(expert_offsets, "expert_offsets", torch.int32, W.shape[0] + 1)
    return rows.shape[0], *W.shape


_PRODUCT_BF16, _PRODUCT_DGRAD, _PRODUCT_WGRAD, _PRODUCT_A4 = 0, 1, 2, 3


def _product_workspace(lib, product, R, E, N, K, device):
    """(tensor that keeps it, pointer, bytes) of a product's workspace; (None, None, 0) where it has none."""
    need = lib.w4a8_grouped_gemm_workspace_bytes(product, R, E, N, K)
    if not need:
        return None, None, 0
    work = torch.empty(need, dtype=torch.uint8, device=device)
    return work, work.data_ptr(), need


def grouped_gemm_bf16(A: torch.Tensor, W: torch.Tensor, expert_offsets: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C bf16 [R, N] of the grouped product with bf16 weights: A bf16 [R, K], W
    bf16 [E, N, K], expert_offsets int32 [E+1].  Rows from offsets[E] on are
    left as `out` holds them, undefined where it is not given."""
    lib = load()
    _bf16(A, "A")
    _bf16(W, "W")
    R, E, N, K = _product(A, W, expert_offsets, 2)
    if out is None:
        out = torch.empty((R, N), dtype=_bfloat16, device=A.device)
    _bf16(out, "out", R * N)
    _here(A, W, expert_offsets, out)
    _keep, work, work_bytes = _product_workspace(lib, _PRODUCT_BF16, R, E, N, K, A.device)
    _check("w4a8_grouped_gemm_bf16", lib.w4a8_grouped_gemm_bf16(
        _ptr(A), _ptr(W), _ptr(expert_offsets), R, E, N, K, _ptr(out), work, work_bytes, _stream()))
    return out


def grouped_gemm_dgrad(dC: torch.Tensor, W: torch.Tensor, expert_offsets: torch.Tensor,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dA bf16 [R, K] of grouped_gemm_bf16 from dC bf16 [R, N] and its W."""
    lib = load()
    _bf16(dC, "dC")
    _bf16(W, "W")
    R, E, N, K = _product(dC, W, expert_offsets, 1)
    if out is None:
        out = torch.empty((R, K), dtype=_bfloat16, device=dC.device)
    _bf16(out, "out", R * K)
    _here(dC, W, expert_offsets, out)
    _keep, work, work_bytes = _product_workspace(lib, _PRODUCT_DGRAD, R, E, N, K, dC.device)
    _check("w4a8_grouped_gemm_dgrad", lib.w4a8_grouped_gemm_dgrad(
        _ptr(dC), _ptr(W), _ptr(expert_offsets), R, E, N, K, _ptr(out), work, work_bytes, _stream()))
    return out


def grouped_gemm_wgrad(dC: torch.Tensor, A: torch.Tensor, expert_offsets: torch.Tensor,
                       out: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """dW [E, N, K] of grouped_gemm_bf16 from dC bf16 [R, N] and its A bf16 [R,
    K]: fp32, or the type of `out` (fp32 or bf16); with accumulate added to what
    `out` holds.  Experts without rows have zeros (nothing added)."""
    lib = load()
    _bf16(dC, "dC")
    _bf16(A, "A")
    if dC.dim() != 2 or A.dim() != 2 or dC.shape[0] != A.shape[0]:
        raise ValueError("dC must be [R, N], A [R, K]")
    R, N = dC.shape
    K = A.shape[1]
    E = expert_offsets.numel() - 1
    _need(expert_offsets, "expert_offsets", torch.int32)
    if out is None:
        if accumulate:
            raise ValueError("accumulate adds to a given out")
        out = torch.empty((E, N, K), dtype=torch.float32, device=dC.device)
    if getattr(out, "dtype", None) is torch.float32:
        _need(out, "out", torch.float32, E * N * K)
    else:
        _bf16(out, "out", E * N * K)
    _here(dC, A, expert_offsets, out)
    _keep, work, work_bytes = _product_workspace(lib, _PRODUCT_WGRAD, R, E, N, K, dC.device)
    _check("w4a8_grouped_gemm_wgrad", lib.w4a8_grouped_gemm_wgrad(
        _ptr(dC), _ptr(A), _ptr(expert_offsets), R, E, N, K, _ptr(out), 0 if out.dtype is torch.float32 else 1,
        int(accumulate), work, work_bytes, _stream()))
    return out


def _fp4_shape(t: torch.Tensor, name: str):
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [N, K] or [E, N, K] (K/2 codes)")
    return (1, *t.shape) if t.dim() == 2 else tuple(t.shape)


def quantize_fp4(w: torch.Tensor, fmt: int, B: Optional[torch.Tensor] = None, SB: Optional[torch.Tensor] = None,
                 expert_scales: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """bf16 weights [E, N, K] (or [N, K], one expert) -> (B uint8 [.., K/2] packed
    E2M1, SB uint8 [.., K/32] E8M0 for fmt WSCALE_MX or [.., K/16] E4M3 for
    WSCALE_NV, expert_scales fp32 [E] for WSCALE_NV, None for WSCALE_MX), as
    grouped_gemm_a16 and matvec take them (MXFP4 also the other products)."""
    lib = load()
    E, N, K = _fp4_shape(w, "w")
    _bf16(w, "w")
    if fmt not in (WSCALE_MX, WSCALE_NV):
        raise ValueError("fmt must be WSCALE_MX or WSCALE_NV")
    if K < 32 or K % 32:
        raise ValueError("K must be a multiple of 32")
    block = 32 if fmt == WSCALE_MX else 16
    if fmt == WSCALE_MX and expert_scales is not None:
        raise ValueError("expert_scales go with WSCALE_NV")
    lead = tuple(w.shape[:-1])
    if B is None:
        B = torch.empty((*lead, K // 2), dtype=torch.uint8, device=w.device)
    if SB is None:
        SB = torch.empty((*lead, K // block), dtype=torch.uint8, device=w.device)
    if fmt == WSCALE_NV and expert_scales is None:
        expert_scales = torch.empty(E, dtype=torch.float32, device=w.device)
    _need(B, "B", torch.uint8, E * N * (K // 2))
    _need(SB, "b_scales", torch.uint8, E * N * (K // block))
    if expert_scales is not None:
        _need(expert_scales, "expert_scales", torch.float32, E)
    need = lib.w4a8_quantize_fp4_bytes(int(fmt), E, N, K)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=w.device)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
    _here(w, B, SB, expert_scales, workspace)
    if E * N:
        _check("w4a8_quantize_fp4", lib.w4a8_quantize_fp4(
            _ptr(w), int(fmt), E, N, K, _ptr(B), _ptr(SB), _ptr(expert_scales), _ptr(workspace),
            0 if workspace is None else workspace.numel(), _stream()))
    elif expert_scales is not None:
        expert_scales.fill_(1.0)   # of experts without weights, as of those of zeros
    return B, SB, expert_scales


def dequantize_fp4(B: torch.Tensor, SB: torch.Tensor, fmt: int, expert_scales: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 weights [.., K] of packed 4-bit ones: B uint8 [E, N, K/2] or [N, K/2],
    SB and expert_scales (fp32 [E] or None for ones) as quantize_fp4 gives them."""
    lib = load()
    E, N, Kh = _fp4_shape(B, "B")
    K = 2 * Kh
    _need(B, "B", torch.uint8)
    if fmt not in (WSCALE_MX, WSCALE_NV):
        raise ValueError("fmt must be WSCALE_MX or WSCALE_NV")
    if K < 32 or K % 32:
        raise ValueError("K must be a multiple of 32")
    _need(SB, "b_scales", torch.uint8, E * N * (K // (32 if fmt == WSCALE_MX else 16)))
    if expert_scales is not None:
        _need(expert_scales, "expert_scales", torch.float32, E)
    if out is None:
        out = torch.empty((*B.shape[:-1], K), dtype=_bfloat16, device=B.device)
    _bf16(out, "out", E * N * K)
    _here(B, SB, expert_scales, out)
    if E * N:
        _check("w4a8_dequantize_fp4", lib.w4a8_dequantize_fp4(
            _ptr(B), _ptr(SB), int(fmt), _ptr(expert_scales), E, N, K, _ptr(out), _stream()))
    return out


def quantize_gather_fp4(x: torch.Tensor, row_of_slot: torch.Tensor, top_k: int, R: int,
                        A: Optional[torch.Tensor] = None, SA: Optional[torch.Tensor] = None):
    """bf16 tokens x [T, K] -> (A uint8 [R, K/2] packed E2M1, SA uint8 [R, K/32]
    E8M0) in the grouped row of every slot (row_of_slot int32 [T * top_k]); rows
    without a slot keep what A and SA hold, zeros where they are not given."""
    lib = load()
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    T, K = x.shape
    _bf16(x, "x")
    if K < 32 or K % 32:
        raise ValueError("K must be a multiple of 32")
    _need(row_of_slot, "row_of_slot", torch.int32, T * top_k)
    if A is None:
        A = torch.zeros((R, K // 2), dtype=torch.uint8, device=x.device)
    if SA is None:
        SA = torch.zeros((R, K // 32), dtype=torch.uint8, device=x.device)
    _need(A, "A", torch.uint8, R * (K // 2))
    _need(SA, "a_scales", torch.uint8, R * (K // 32))
    _here(x, row_of_slot, A, SA)
    _check("w4a8_quantize_gather_fp4", lib.w4a8_quantize_gather_fp4(
        _ptr(x), T, K, _ptr(row_of_slot), int(top_k), int(R), _ptr(A), _ptr(SA), _stream()))
    return A, SA


def grouped_gemm_a4(A: torch.Tensor, SA: torch.Tensor, B: torch.Tensor, SB: torch.Tensor,
                    expert_offsets: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C bf16 [R, N] of the grouped product of MXFP4 rows and weights: A uint8
    [R, K/2], SA uint8 [R, K/32], B uint8 [E, N, K/2], SB uint8 [E, N, K/32],
    expert_offsets int32 [E+1].  Rows from offsets[E] on are left as `out` holds
    them, undefined where it is not given."""
    lib = load()
    if A.dim() != 2 or B.dim() != 3 or SB.dim() != 3:
        raise ValueError("A must be [R, K/2], B [E, N, K/2], SB [E, N, K/32]")
    R, Kh = A.shape
    E, N, K = B.shape[0], B.shape[1], 2 * B.shape[2]
    if 2 * Kh != K or SB.shape != (E, N, K // 32):
        raise ValueError("inconsistent K between A, B and SB")
    _need(A, "A", torch.uint8)
    _need(SA, "a_scales", torch.uint8, R * (K // 32))
    _need(B, "B", torch.uint8)
    _need(SB, "b_scales", torch.uint8)
    _need(expert_offsets, "expert_offsets", torch.int32, E + 1)
    if out is None:
        out = torch.empty((R, N), dtype=_bfloat16, device=A.device)
    _bf16(out, "out", R * N)
    _here(A, SA, B, SB, expert_offsets, out)
    _keep, work, work_bytes = _product_workspace(lib, _PRODUCT_A4, R, E, N, K, A.device)
    _check("w4a8_grouped_gemm_a4", lib.w4a8_grouped_gemm_a4(
        _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(expert_offsets), R, E, N, K, _ptr(out), work, work_bytes, _stream()))
    return out


_GRAD_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def _grad_list(tensors, name, like=None):
    """(pointers, elements, types) of a list of tensors.  Each property of all at a time: this is most of a small
    call's time (40 tensors and their outputs: 29 us a call, 36 with one tensor tested after the other)."""
    dev = _current_device()
    if not all(isinstance(t, _Tensor) for t in tensors):
        raise TypeError(f"{name}s must be torch tensors")
    kinds = [_GRAD_TYPES.get(t.dtype) for t in tensors]
    numel = list(map(_Tensor.numel, tensors))
    if None in kinds or (like is not None and kinds != like[2]):
        bad = next(i for i, k in enumerate(kinds) if k is None or (like is not None and k != like[2][i]))
        raise TypeError(f"{name} {bad} must be " + ("float32 or bfloat16" if like is None else "of its tensor's type") +
                        f", got {tensors[bad].dtype}")
    if any(map(dev.__ne__, map(_Tensor.get_device, tensors))):
        raise ValueError(f"every {name} must be on the current device (cuda:{dev})")
    if not all(map(_Tensor.is_contiguous, tensors)):
        raise ValueError(f"every {name} must be contiguous")
    if like is not None and numel != like[1]:
        raise ValueError(f"every {name} must have as many elements as its tensor")
    return list(map(_Tensor.data_ptr, tensors)), numel, kinds


def _grads(tensors, outs, max_norm, eps, norm, workspace):
    lib = load()
    n = len(tensors)
    found = _grad_list(tensors, "tensor")
    if outs is None or outs is tensors:
        optrs = found[0]
    else:
        if len(outs) != n:
            raise ValueError(f"out must hold {n} tensors, got {len(outs)}")
        optrs = _grad_list(outs, "out", found)[0]
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=torch.device("cuda", _current_device()))
    _need(norm, "norm", torch.float32, 1)
    # array.array: a third of the time of a ctypes array (40 tensors: 32 us a call with those)
    ptrs, numel, kinds = array("Q", found[0]), array("q", found[1]), array("i", found[2])
    optrs = None if outs is None else array("Q", optrs)
    at_numel = numel.buffer_info()[0]
    if workspace is None:
        workspace = torch.empty(lib.w4a8_clip_grads_bytes(at_numel, n), dtype=torch.uint8, device=norm.device)
    _need(workspace, "workspace", torch.uint8)
    _here(norm, workspace)
    _check("w4a8_clip_grads", lib.w4a8_clip_grads(
        ptrs.buffer_info()[0], None if outs is None else optrs.buffer_info()[0], at_numel, kinds.buffer_info()[0], n,
        float(max_norm), float(eps), _ptr(workspace), workspace.numel(), _ptr(norm), _stream()))
    return norm


def grad_norm(tensors, norm: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """norm fp32 [1] = sqrt of the sum of all squares of a list of contiguous fp32
    and bf16 tensors, summed in 64 bits."""
    return _grads(list(tensors), None, 0.0, 0.0, norm, workspace)


def clip_grads(tensors, max_norm: float, eps: float = 1e-6, out=None, norm: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scale a list of contiguous fp32 and bf16 tensors by min(1, max_norm /
    (norm + eps)), norm that of them all (grad_norm), and return the norm, fp32
    [1].  In place, or into the tensors of the list `out`; no tensor may be in
    the list twice."""
    tensors = list(tensors)
    return _grads(tensors, tensors if out is None else list(out), max_norm, eps, norm, workspace)
