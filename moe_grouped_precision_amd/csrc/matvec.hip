// Products of single tokens with 4-bit weights and group scales, gfx950:
//
//   y[s, n] = bf16( gs[e] * sum_k x[row(s), k] * (q(e, n, k) - z(e, n, k / g)) * s(e, n, k / g) )
//
// e = the slot's expert (0 without ids), row(s) = s / (S / X).  MXFP4: q an
// E2M1 value, s = 2^(code - 127) per 32 K; NVFP4: s an E4M3 value per 16 K;
// INT4: q a code 0 .. 15, z its zero point (8 when none are given), s bf16
// per 32, 64 or 128 K.  No zero point for the first two.
//
// One wave per (slot, column).
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

namespace w4a8 {
namespace {

typedef float v2f __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float e2m1(uint32_t c) {
  const float mag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  const float v = mag[c & 7];
  return (c & 8) ? -v : v;
}

template <int FMT>
__device__ __forceinline__ float group_scale(const void* p, size_t i) {
  if (FMT == 0) {
    const uint32_t c = ((const uint8_t*)p)[i];
    return c == 0xff ? __builtin_nanf("") : c == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(c << 23);
  }
  if (FMT == 1) return __builtin_amdgcn_cvt_pk_f32_fp8((int)((const uint8_t*)p)[i], false)[0];
  return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}

template <int FMT>
__global__ void __launch_bounds__(256)
matvec_kernel(const uint16_t* __restrict__ x, int per_row, const uint8_t* __restrict__ B, const void* __restrict__ SB,
              int group, const uint8_t* __restrict__ zeros, const float* __restrict__ gs,
              const int32_t* __restrict__ ids, int E, int N, int K, uint16_t* __restrict__ y) {
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int s = blockIdx.y;
  if (n >= N) return;
  const int e = ids ? ids[s] : 0;
  float acc = 0.f;
  if (e >= 0 && e < E) {
    const size_t col = (size_t)e * N + n;
    const uint16_t* xr = x + (size_t)(s / per_row) * K;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(B + col * (size_t)(K >> 1));
    for (int c = lane; c < K / 8; c += 64) {  // 8 weights: inside one group
      const size_t gi = col * (size_t)(K / group) + (8 * c) / group;
      const float sc = group_scale<FMT>(SB, gi);
      const float z = FMT != 2 ? 0.f : zeros ? (float)zeros[gi] : 8.f;
      const uint32_t v = w[c];
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t q = (v >> (4 * i)) & 15u;
        part = fmaf(__uint_as_float((uint32_t)xr[8 * c + i] << 16), FMT == 2 ? (float)q - z : e2m1(q), part);
      }
      acc = fmaf(part, sc, acc);
    }
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) acc += __shfl_xor(acc, i, 64);
    if (gs) acc *= gs[e];
  }
  if (lane == 0) y[(size_t)s * N + n] = __builtin_bit_cast(uint16_t, (__bf16)acc);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream) {
  const dim3 grid((a.N + 3) / 4, a.S), block(256);
  const int per_row = a.S / a.X;
  if (a.fmt == 0)
    hipLaunchKernelGGL(matvec_kernel<0>, grid, block, 0, stream, a.x, per_row, a.B, a.SB, 32, a.zeros, a.gs, a.ids,
                       a.E, a.N, a.K, a.y);
  else if (a.fmt == 1)
    hipLaunchKernelGGL(matvec_kernel<1>, grid, block, 0, stream, a.x, per_row, a.B, a.SB, 16, a.zeros, a.gs, a.ids,
                       a.E, a.N, a.K, a.y);
  else
    hipLaunchKernelGGL(matvec_kernel<2>, grid, block, 0, stream, a.x, per_row, a.B, a.SB, a.group, a.zeros, a.gs,
                       a.ids, a.E, a.N, a.K, a.y);
  return hipGetLastError();
}

}  // namespace w4a8
