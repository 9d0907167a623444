// Host-side launch interface between the C ABI layer (api.cpp) and the kernel
// translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a8 {

struct GemmArgs {
  const uint8_t* A;        // [R][K] E4M3 codes
  const float* SA;         // per (row, 128-K group), layout below
  const uint8_t* B;        // [E][N][K/2] packed E2M1
  const uint8_t* SB;       // [E][N][K/32] E8M0
  const int32_t* offsets;  // [E+1]
  uint16_t* C;             // [R][N] bf16 bits (the plain GEMM)
  int E, N, K, layout;     // layout 0 row-major, 1 M-major
  // fused SwiGLU epilogue (N = 2 I weight columns: gate 0 .. I-1, up I .. 2I-1)
  uint8_t* A2;             // [R][I] E4M3 codes of silu(gate) * up
  float* SA2;              // per (row, 128 columns of A2), layout2
  int I, layout2;
  // planned GEMM: a tile list in w4a8_plan's format holding at most max_tiles tiles
  const int32_t* plan;
  int max_tiles;
};

// Route prep: the workgroup holds up to ROUTE_MAX_WAVES waves, W of which
// rank (1..ROUTE_MAX_WAVES), and route_prep_lds_bytes(E, W) bytes of LDS;
// route_prep_waves picks the largest W that fits lds_limit bytes, 0 if none
// does, and the launch lowers W (and the waves) for batches of few ids.
constexpr int ROUTE_MAX_WAVES = 16;
constexpr int ROUTE_LOADS = 16;  // 16-byte id loads in flight per lane
size_t route_prep_lds_bytes(int E, int waves);
int route_prep_waves(int E, size_t lds_limit);
hipError_t launch_route_prep(const int32_t* ids, int n, int E, int W, int32_t* counts, int32_t* offsets,
                             int32_t* row_of_slot, hipStream_t stream);
hipError_t launch_plan(const int32_t* offsets, int E, int N, int32_t* plan, int max_tiles,
                       hipStream_t stream);
hipError_t launch_grouped_gemm(const GemmArgs& args, int grid, hipStream_t stream);
hipError_t launch_grouped_gemm_swiglu(const GemmArgs& args, int grid, hipStream_t stream);
hipError_t launch_grouped_gemm_planned(const GemmArgs& args, int grid, hipStream_t stream);
hipError_t grouped_gemm_occupancy(int* blocks);
hipError_t launch_combine(const uint16_t* C, int R, int N, const int32_t* row_of_slot, const float* weights, int T,
                          int top_k, uint16_t* out, hipStream_t stream);
hipError_t launch_swiglu_quant(const uint16_t* C, int R, int I, uint8_t* A, float* SA, int layout,
                               hipStream_t stream);
hipError_t launch_grouped_gemm_a16(const uint16_t* A, const uint8_t* B, const uint8_t* SB, int fmt, const float* GS,
                                   const int32_t* offsets, int E, int N, int K, uint16_t* C, int grid,
                                   hipStream_t stream);
hipError_t launch_quant_gather(const uint16_t* x, int T, int K, const int32_t* row_of_slot, int top_k, int R,
                               uint8_t* A, float* SA, int layout, hipStream_t stream);

// A launch may have fewer than 2^32 threads per dimension; one with more is
// cut to their number modulo 2^32, without an error.  n items of `threads`
// threads each therefore go in as many launches as it takes: launch(first
// item, number of items), half the limit at most in one.
constexpr int64_t MAX_THREADS = (int64_t)1 << 31;
template <typename F>
hipError_t in_launches(int64_t n, int64_t threads, F launch) {
  const int64_t most = MAX_THREADS / threads;
  for (int64_t i = 0; i < n; i += most) {
    launch(i, n - i < most ? n - i : most);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_topk_gate(const void* logits, bool bf16, int T, int E, int k, int score, int renorm, float scale,
                            int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_topk_gate_backward(const void* logits, bool bf16, int T, int E, const int32_t* ids,
                                     const float* dweights, int k, int score, int renorm, float scale, void* dlogits,
                                     hipStream_t stream);
hipError_t launch_dispatch(const uint16_t* x, int T, int K, const int32_t* row_of_slot, int top_k, int R, uint16_t* A,
                           hipStream_t stream);
hipError_t launch_dispatch_backward(const uint16_t* dA, int R, int K, const int32_t* row_of_slot, int T, int top_k,
                                    uint16_t* dx, hipStream_t stream);
hipError_t launch_combine_backward(const uint16_t* C, const uint16_t* dout, int R, int N, const int32_t* row_of_slot,
                                   const float* weights, int T, int top_k, uint16_t* dC, float* dweights,
                                   hipStream_t stream);

struct MatvecArgs {
  const uint16_t* x;       // [X][K] bf16
  const uint8_t* B;        // [E][N][K/2] 4-bit codes
  const void* SB;          // [E][N][K/group]
  const uint8_t* zeros;    // [E][N][K/group] or null
  const float* gs;         // [E] or null
  const int32_t* ids;      // [S] or null (E = 1)
  uint16_t* y;             // [S][N] bf16
  int S, E, N, K, fmt, group;
  int per_row_inv;         // slot s multiplies row (s * per_row_inv) >> 16 of x (s < 64)
  // bytes of a column and of an expert (the path needs an expert's weights below 2^32 bytes)
  uint32_t wcol, scol, zcol, wexp, sexp, zexp;
};
hipError_t launch_matvec(const MatvecArgs& args, int cus, hipStream_t stream);
hipError_t launch_swiglu(const uint16_t* C, int R, int I, uint16_t* h, uint8_t* codes, float* scales,
                         hipStream_t stream);
hipError_t launch_swiglu_backward(const uint8_t* codes, const float* scales, const uint16_t* dh, int R, int I,
                                  uint16_t* dC, uint16_t* h, hipStream_t stream);

}  // namespace w4a8
