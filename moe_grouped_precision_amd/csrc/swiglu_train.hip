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
// A stream: 16 lanes per 128 columns of g and the same of u, 8 columns of each
// per lane (16-byte loads, consecutive lanes), the group maxima by DPP
// rotations; no LDS, no barrier.  Bound by HBM's mix of reads and writes: 9216
// rows of I = 2048 with the copy 26.0 us in the kernel (152 MB: 5.8 TB/s), the
// gradient with h 32.7 us (190 MB: 5.8 TB/s); a plain copy of large buffers
// runs at 4.7.  I = 2176, whose rows take a workgroup of 16 groups and one of
// a single group: 39 and 47 us a call (4.1 and 4.3 TB/s).  8 lanes per group with two loads each took 30.6 and 37.7 us,
// a 64-bit division per lane 1% more.
#include "swiglu.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

namespace w4a8 {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kCkptFloor = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
  const v4u a = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(a[i] << 16);
    f[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  v4u a;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * i], f[2 * i + 1]}, v2bf));
  __builtin_nontemporal_store(a, reinterpret_cast<v4u*>(p));
}

// Maximum over 16 lanes, in each of them.
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
  return fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float max16(float v) {
  v = max_dpp<0x128>(v);   // row_ror 8, 4, 2, 1
  v = max_dpp<0x124>(v);
  v = max_dpp<0x122>(v);
  return max_dpp<0x121>(v);
}

// The 8-bit copy of one lane's 8 columns; the group's 16 lanes agree on the
// scale.  No clip: |f / q| stays under 448 (1 + 2^-8), which rounds to 448; a
// NaN keeps its NaN code, an infinity makes the group's scale infinite and
// the group NaN when it is read.
__device__ __forceinline__ void quant8(const float (&f)[8], uint8_t* codes, float* scale, bool write_scale) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  m = max16(m);
  const float q = m < kCkptFloor ? 1.0f : __fdiv_rn(m, 448.0f);
  const float inv = __fdiv_rn(1.0f, q);
  v2u c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, w, true);
    c[i] = (uint32_t)w;
  }
  __builtin_nontemporal_store(c, reinterpret_cast<v2u*>(codes));
  if (write_scale) *scale = q;
}

constexpr int S_GROUPS = 16;   // most groups of a workgroup

template <bool CKPT>
__global__ void __launch_bounds__(16 * S_GROUPS)
swiglu_kernel(const uint16_t* __restrict__ C, int blocks, int I, uint16_t* __restrict__ h,
              uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int G = I >> 7;
  const int lane = threadIdx.x & 15;
  const uint32_t r = blockIdx.x / (uint32_t)blocks;   // blocks: workgroups of a row
  const int g = (int)(blockIdx.x - r * blocks) * (int)(blockDim.x >> 4) + (int)(threadIdx.x >> 4);
  if (g >= G) return;
  const size_t at = (size_t)r * 2 * I + g * 128 + lane * 8;
  float fg[8], fu[8], fh[8];
  load8(C + at, fg);
  load8(C + at + I, fu);
#pragma unroll
  for (int e = 0; e < 8; ++e) fh[e] = swiglu_f32(fg[e], fu[e]);
  store8(h + (size_t)r * I + g * 128 + lane * 8, fh);
  if (CKPT) {
    quant8(fg, codes + at, scales + (size_t)r * 2 * G + g, lane == 0);
    quant8(fu, codes + at + I, scales + (size_t)r * 2 * G + G + g, lane == 0);
  }
}

__device__ __forceinline__ void decode8(const uint8_t* p, float (&f)[8]) {
  const v2u c = __builtin_nontemporal_load(reinterpret_cast<const v2u*>(p));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    f[4 * i] = a[0];
    f[4 * i + 1] = a[1];
    f[4 * i + 2] = b[0];
    f[4 * i + 3] = b[1];
  }
}

template <bool WITH_H>
__global__ void __launch_bounds__(16 * S_GROUPS)
swiglu_backward_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                       const uint16_t* __restrict__ dh, int blocks, int I, uint16_t* __restrict__ dC,
                       uint16_t* __restrict__ h) {
  const int G = I >> 7;
  const int lane = threadIdx.x & 15;
  const uint32_t r = blockIdx.x / (uint32_t)blocks;   // blocks: workgroups of a row
  const int g = (int)(blockIdx.x - r * blocks) * (int)(blockDim.x >> 4) + (int)(threadIdx.x >> 4);
  if (g >= G) return;
  const size_t at = (size_t)r * 2 * I + g * 128 + lane * 8;
  const size_t hat = (size_t)r * I + g * 128 + lane * 8;
  float fg[8], fu[8], fd[8];
  const float qg = scales[(size_t)r * 2 * G + g], qu = scales[(size_t)r * 2 * G + G + g];
  decode8(codes + at, fg);
  decode8(codes + at + I, fu);
  load8(dh + hat, fd);
  float dg[8], du[8], hh[8], slope[8], most = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // g = code * q needs 28 bits: what fp32 cuts off it (lo) would cost |g|
    // times its size in e^-g, so e^-(g + lo) = e^-g (1 - lo) where |g| < 104
    // (there |lo| <= 2^-18; for larger gates lo reaches 1 and more, and s is
    // 0 or 1 without it).  e^-g is capped at e^88, where it and its reciprocal
    // stay finite; from -104 down s is below half of fp32's smallest value and
    // taken as 0, or g s would grow with |g|.
    const float gv = fg[e] * qg, lo = fmaf(fg[e], qg, -gv), uv = fu[e] * qu;
    const float x0 = exp_f32(fminf(-gv, 88.0f));
    const float x = fabsf(gv) < 104.0f ? fmaf(-x0, lo, x0) : x0;
    const float s = gv <= -104.0f ? 0.0f : __builtin_amdgcn_rcpf(1.0f + x);
    const float silu = gv * s, prod = fd[e] * uv;
    slope[e] = s * fmaf(gv, x * s, 1.0f);
    most = fmaxf(most, fabsf(prod));
    dg[e] = prod * slope[e];
    du[e] = fd[e] * silu;
    hh[e] = silu * uv;
  }
  // dh u first (u slope may underflow under a large dh); where that left fp32,
  // slope (at most 1.1) goes in between
  if (__builtin_expect(most == __builtin_inff(), 0)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[e] = fabsf(fd[e] * (fu[e] * qu)) < __builtin_inff() ? dg[e] : fd[e] * (fu[e] * qu * slope[e]);
  }
  store8(dC + at, dg);
  store8(dC + at + I, du);
  if (WITH_H) store8(h + hat, hh);
}

}  // namespace

hipError_t launch_swiglu(const uint16_t* C, int R, int I, uint16_t* h, uint8_t* codes, float* scales,
                         hipStream_t stream) {
  const int G = I >> 7, blocks = (G + S_GROUPS - 1) / S_GROUPS;
  const int threads = 16 * (G < S_GROUPS ? G : S_GROUPS);
  return in_launches(R, (int64_t)blocks * threads, [&](int64_t r, int64_t n) {
    const dim3 grid((unsigned)(n * blocks)), block(threads);
    const uint16_t* c = C + r * 2 * I;
    if (codes)
      hipLaunchKernelGGL(swiglu_kernel<true>, grid, block, 0, stream, c, blocks, I, h + r * I, codes + r * 2 * I,
                         scales + r * 2 * G);
    else
      hipLaunchKernelGGL(swiglu_kernel<false>, grid, block, 0, stream, c, blocks, I, h + r * I, codes, scales);
  });
}

hipError_t launch_swiglu_backward(const uint8_t* codes, const float* scales, const uint16_t* dh, int R, int I,
                                  uint16_t* dC, uint16_t* h, hipStream_t stream) {
  const int G = I >> 7, blocks = (G + S_GROUPS - 1) / S_GROUPS;
  const int threads = 16 * (G < S_GROUPS ? G : S_GROUPS);
  return in_launches(R, (int64_t)blocks * threads, [&](int64_t r, int64_t n) {
    const dim3 grid((unsigned)(n * blocks)), block(threads);
    const uint8_t* q = codes + r * 2 * I;
    const float* s = scales + r * 2 * G;
    if (h)
      hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, block, 0, stream, q, s, dh + r * I, blocks, I,
                         dC + r * 2 * I, h + r * I);
    else
      hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, block, 0, stream, q, s, dh + r * I, blocks, I,
                         dC + r * 2 * I, h);
  });
}

}  // namespace w4a8
