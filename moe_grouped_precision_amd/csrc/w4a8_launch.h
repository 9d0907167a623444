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

struct NormArgs {
  const uint16_t* x;       // [T][K] bf16
  const uint16_t* res;     // [T][K] or null
  const void* w;           // [K] bf16 or fp32, or null (ones)
  uint16_t* y;             // [T][K] or null
  uint16_t* h;             // [T][K] x + res, or null
  uint8_t* A;              // [T][K] E4M3 codes of y, or null
  float* SA;               // per (row, 128 columns), layout 0 row-major, 1 M-major
  int T, K, w_f32, layout;
  float eps;
};
struct NormGradArgs {
  const uint16_t* h;       // [T][K]
  const uint16_t* dy;      // [T][K]
  const uint16_t* dres;    // [T][K] or null
  const void* w;           // [K] or null
  uint16_t* dx;            // [T][K]
  float* dw;               // [K] or null
  float* partials;         // [norm_backward_parts(T)][K]
  int T, K, w_f32;
  float eps;
};
constexpr int NORM_PARTS = 512;   // most workgroups of the gradient, each with a part of dw
int norm_backward_parts(int T);
hipError_t launch_rms_norm(const NormArgs& args, hipStream_t stream);
hipError_t launch_rms_norm_backward(const NormGradArgs& args, hipStream_t stream);

// Gradient norm: workgroups of a launch at most, each with one partial sum; the
// workspace holds grad_norm_parts() + 1 of them.
constexpr int GN_GRID = 1024;
int grad_norm_parts(const int64_t* numel, int n);
hipError_t launch_clip_grads(const void* const* in, void* const* out, const int64_t* numel, const int* types, int n,
                             float max_norm, float eps, double* partials, float* norm, hipStream_t stream);

size_t quant_fp4_workspace(bool nv, int E, int N, int K);
hipError_t launch_quant_fp4(const uint16_t* x, bool nv, int E, int N, int K, uint8_t* B, uint8_t* SB, float* gs,
                            uint32_t* work, hipStream_t stream);
hipError_t launch_dequant_fp4(const uint8_t* B, const uint8_t* SB, bool nv, const float* gs, int E, int N, int K,
                              uint16_t* out, hipStream_t stream);
hipError_t launch_quant_gather_fp4(const uint16_t* x, int T, int K, const int32_t* row_of_slot, int top_k, int R,
                                   uint8_t* A, uint8_t* SA, hipStream_t stream);

// The tiled products out[y, x] = sum over z: rows (or N of the weights' gradient)
// along y, weights (or K) along x.
struct TileArgs {
  const uint8_t* Y;        // A, dC: rows
  const uint8_t* X;        // W, or A for the weights' gradient
  const uint8_t* SY;       // E8M0 codes of FP4 rows [R][K/32] and weights [E][N][K/32]
  const uint8_t* SX;
  const int32_t* offsets;  // [E+1]
  void* out;
  int E, R, N, K, accumulate;
  int slices, wide;        // of z; outputs in whole 16 bytes (both set at the launch)
};
enum { PRODUCT_FWD = 0, PRODUCT_ROWS = 1, PRODUCT_WEIGHTS = 2, PRODUCT_FOUR = 3 };
// Slices of a product's sum, and the bytes of their parts (0 for one slice).
int product_slices(int product, int R, int E, int N, int K);
size_t product_workspace(int product, int R, int E, int N, int K);
// Its tile, rows << 16 | columns, for operands at 16-byte alignment.
int product_tile(int product, int R, int E, int N, int K);
// work: product_workspace() bytes, or null for one slice in any case
hipError_t launch_grouped_bf16(const TileArgs& args, void* work, hipStream_t stream);
hipError_t launch_grouped_dgrad(const TileArgs& args, void* work, hipStream_t stream);
hipError_t launch_grouped_wgrad(const TileArgs& args, bool f32, void* work, hipStream_t stream);
hipError_t launch_grouped_a4(const TileArgs& args, void* work, hipStream_t stream);

}  // namespace w4a8
