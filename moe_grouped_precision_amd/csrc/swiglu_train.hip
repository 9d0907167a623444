// SwiGLU in bf16 with an 8-bit copy of its input, and the backward pass from
// that copy, gfx950.
//
//   h = silu(g) u,  g = C[:, :I], u = C[:, I:],  silu(g) = g s, s = 1 / (1 + e^-g)
//   copy: per (row, 128 columns of C), a = max|C|, q = a / 448 (1 where a <
//         2^-100), code = E4M3(C * (1 / q))
//   backward, from g, u = code * q:
//         dg = dh u s (1 + g (1 - s)),  du = dh g s,  h = g s u
// fp32 throughout, one rounding to bf16 per output.
//
// A stream: 8 lanes per 128 columns of g and the same of u, 16 columns of
// each per lane, the group maxima by three lane exchanges; no LDS, no barrier.
#include "swiglu.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

namespace w4a8 {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kCkptFloor = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ void load16(const uint16_t* p, float (&f)[16]) {
  const v4u a = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  const v4u b = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p) + 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(a[i] << 16);
    f[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    f[8 + 2 * i] = __uint_as_float(b[i] << 16);
    f[8 + 2 * i + 1] = __uint_as_float(b[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store16(uint16_t* p, const float (&f)[16]) {
  v4u a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * i], f[2 * i + 1]}, v2bf));
    b[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[8 + 2 * i], f[8 + 2 * i + 1]}, v2bf));
  }
  __builtin_nontemporal_store(a, reinterpret_cast<v4u*>(p));
  __builtin_nontemporal_store(b, reinterpret_cast<v4u*>(p) + 1);
}

// The 8-bit copy of one lane's 16 columns; the group's 8 lanes agree on the
// scale.  No clip: |f / q| stays under 448 (1 + 2^-8), which rounds to 448; a
// NaN keeps its NaN code, an infinity makes the group's scale infinite and
// the group NaN when it is read.
__device__ __forceinline__ void quant16(const float (&f)[16], uint8_t* codes, float* scale, bool write_scale) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
  m = fmaxf(m, __shfl_xor(m, 1, 8));
  m = fmaxf(m, __shfl_xor(m, 2, 8));
  m = fmaxf(m, __shfl_xor(m, 4, 8));
  const float q = m < kCkptFloor ? 1.0f : __fdiv_rn(m, 448.0f);
  const float inv = __fdiv_rn(1.0f, q);
  v4u c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, w, true);
    c[i] = (uint32_t)w;
  }
  __builtin_nontemporal_store(c, reinterpret_cast<v4u*>(codes));
  if (write_scale) *scale = q;
}

template <bool CKPT>
__global__ void __launch_bounds__(256)
swiglu_kernel(const uint16_t* __restrict__ C, int64_t groups, int I, uint16_t* __restrict__ h,
              uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int G = I >> 7;
  const int lane8 = threadIdx.x & 7;
  const int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  if (i >= groups) return;
  const int64_t r = i / G;
  const int g = (int)(i - r * G);
  const size_t at = (size_t)r * 2 * I + g * 128 + lane8 * 16;
  float fg[16], fu[16], fh[16];
  load16(C + at, fg);
  load16(C + at + I, fu);
#pragma unroll
  for (int e = 0; e < 16; ++e) fh[e] = swiglu_f32(fg[e], fu[e]);
  store16(h + (size_t)r * I + g * 128 + lane8 * 16, fh);
  if (CKPT) {
    quant16(fg, codes + at, scales + (size_t)r * 2 * G + g, lane8 == 0);
    quant16(fu, codes + at + I, scales + (size_t)r * 2 * G + G + g, lane8 == 0);
  }
}

__device__ __forceinline__ void decode16(const uint8_t* p, float (&f)[16]) {
  const v4u c = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    f[4 * i] = a[0];
    f[4 * i + 1] = a[1];
    f[4 * i + 2] = b[0];
    f[4 * i + 3] = b[1];
  }
}

template <bool WITH_H>
__global__ void __launch_bounds__(256)
swiglu_backward_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                       const uint16_t* __restrict__ dh, int64_t groups, int I, uint16_t* __restrict__ dC,
                       uint16_t* __restrict__ h) {
  const int G = I >> 7;
  const int lane8 = threadIdx.x & 7;
  const int64_t i = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  if (i >= groups) return;
  const int64_t r = i / G;
  const int g = (int)(i - r * G);
  const size_t at = (size_t)r * 2 * I + g * 128 + lane8 * 16;
  const size_t hat = (size_t)r * I + g * 128 + lane8 * 16;
  float fg[16], fu[16], fd[16];
  const float qg = scales[(size_t)r * 2 * G + g], qu = scales[(size_t)r * 2 * G + G + g];
  decode16(codes + at, fg);
  decode16(codes + at + I, fu);
  load16(dh + hat, fd);
  float dg[16], du[16], hh[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    // g = code * q needs 28 bits: what fp32 cuts off it (lo) would cost |g|
    // times its size in e^-g, so e^-(g + lo) = e^-g (1 - lo).  e^-g is capped
    // at e^88, where it and its reciprocal stay finite.
    const float gv = fg[e] * qg, lo = fmaf(fg[e], qg, -gv), uv = fu[e] * qu;
    const float x0 = exp_f32(fminf(-gv, 88.0f));
    const float x = fmaf(-x0, lo, x0);
    const float s = __builtin_amdgcn_rcpf(1.0f + x);
    const float silu = gv * s;
    dg[e] = fd[e] * uv * (s * fmaf(gv, x * s, 1.0f));
    du[e] = fd[e] * silu;
    hh[e] = silu * uv;
  }
  store16(dC + at, dg);
  store16(dC + at + I, du);
  if (WITH_H) store16(h + hat, hh);
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* C, int R, int I, uint16_t* h, uint8_t* codes, float* scales,
                         hipStream_t stream) {
  const int64_t groups = (int64_t)R * (I >> 7);
  const dim3 grid((unsigned)((groups + 31) / 32));
  if (codes)
    hipLaunchKernelGGL(swiglu_kernel<true>, grid, dim3(256), 0, stream, C, groups, I, h, codes, scales);
  else
    hipLaunchKernelGGL(swiglu_kernel<false>, grid, dim3(256), 0, stream, C, groups, I, h, codes, scales);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const uint8_t* codes, const float* scales, const uint16_t* dh, int R, int I,
                                  uint16_t* dC, uint16_t* h, hipStream_t stream) {
  const int64_t groups = (int64_t)R * (I >> 7);
  const dim3 grid((unsigned)((groups + 31) / 32));
  if (h)
    hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, dim3(256), 0, stream, codes, scales, dh, groups, I, dC, h);
  else
    hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, dim3(256), 0, stream, codes, scales, dh, groups, I, dC, h);
  return hipGetLastError();
}

}  // namespace w4a8
