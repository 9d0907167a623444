// The norm of many tensors as one vector, and their scaling by it, gfx950.
//
//   norm = sqrt(sum over all tensors of x^2),
//   c = min(1, max_norm / (norm + eps)),  out = round(c x) in the tensor's type
//
// A launch takes up to GN_TENSORS tensors in its arguments (no table in device
// memory to fill, nothing of it left for the next call, and a captured graph
// holds them like any pointer), cut into chunks of GN_CHUNK elements that its
// workgroups take in turn.  Squares and sums are in 64 bits: no gradient is too
// large or too small for its square, and the conversions hide behind HBM.
// Every workgroup leaves one partial sum in the workspace; they are added in a
// fixed order, so the result does not change from run to run.
//
// Bound by HBM: 1057 MB of gradients, norm 173 us (6.1 TB/s), clipping 341 (6.2).
// 1024 workgroups, four waves to a SIMD (2048: 595 us for both in place of 564, 768:
// 566, 512: 634; twice the loads of a thread: 580).  Small lists: 40 tensors of up
// to 300000 elements 4.6 and 6.4 us, their call 29 by the host's work.
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace w4a8 {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int GN_TENSORS = 96;       // of a launch: 28 bytes each, under the 4 KB of kernel arguments
constexpr int GN_CHUNK = 8192;       // elements: 4 or 8 loads of 16 bytes per thread
constexpr int GN_THREADS = 256;

struct Tensors {
  const void* in[GN_TENSORS];
  void* out[GN_TENSORS];
  int64_t numel[GN_TENSORS];
  uint32_t first[GN_TENSORS];   // the tensor's first chunk
  uint32_t f32[GN_TENSORS / 32];
  uint32_t n, chunks;
};

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The tensor of a chunk: the last one that starts at or before it (wave-uniform).
__device__ __forceinline__ int tensor_of(const Tensors& t, uint32_t chunk) {
  int lo = 0, hi = (int)t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double a = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) a += s[w];
  return a;
}

__global__ void __launch_bounds__(GN_THREADS)
square_sum_kernel(const Tensors t, double* __restrict__ partials) {
  __shared__ double s[GN_THREADS / 64];
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (int64_t)(c - t.first[i]) * GN_CHUNK;
    const int n = (int)(t.numel[i] - at < GN_CHUNK ? t.numel[i] - at : GN_CHUNK);
    int done = 0;
    if ((t.f32[i >> 5] >> (i & 31)) & 1u) {
      const float* p = static_cast<const float*>(t.in[i]) + at;
      if (aligned16(p)) {
        done = n & ~3;
#pragma unroll 4
        for (int e = threadIdx.x * 4; e < done; e += GN_THREADS * 4) {
          const v4u v = *reinterpret_cast<const v4u*>(p + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double x = (double)__uint_as_float(v[j]);
            acc[j] = fma(x, x, acc[j]);
          }
        }
      }
      for (int e = done + threadIdx.x; e < n; e += GN_THREADS) {
        const double x = (double)p[e];
        acc[0] = fma(x, x, acc[0]);
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(t.in[i]) + at;
      if (aligned16(p)) {
        done = n & ~7;
#pragma unroll 4
        for (int e = threadIdx.x * 8; e < done; e += GN_THREADS * 8) {
          const v4u v = *reinterpret_cast<const v4u*>(p + e);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double x = (double)__uint_as_float(v[j] << 16), y = (double)__uint_as_float(v[j] & 0xffff0000u);
            acc[j] = fma(x, x, acc[j]);
            acc[j] = fma(y, y, acc[j]);
          }
        }
      }
      for (int e = done + threadIdx.x; e < n; e += GN_THREADS) {
        const double x = (double)__uint_as_float((uint32_t)p[e] << 16);
        acc[0] = fma(x, x, acc[0]);
      }
    }
  }
  const double v = block_sum((acc[0] + acc[1]) + (acc[2] + acc[3]), s);
  if (threadIdx.x == 0) partials[blockIdx.x] = v;
}

// The partial sums' sum, the same bits in every workgroup that asks.
__device__ __forceinline__ double sum_of(const double* partials, int parts, double* s) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += GN_THREADS) v += partials[i];
  return block_sum(v, s);
}

// The norm by itself; the whole sum also goes behind the partial ones.
__global__ void __launch_bounds__(GN_THREADS)
norm_kernel(double* partials, int parts, float* __restrict__ norm) {
  __shared__ double s[GN_THREADS / 64];
  const double v = sum_of(partials, parts, s);
  if (threadIdx.x == 0) {
    partials[parts] = v;
    *norm = (float)sqrt(v);
  }
}

// min(1, ratio) as c * d.  d is 1 where fp32 holds c whole; below, where norms are
// 2^126 times max_norm and more (fp32 alone left c fewer bits there, and 0 below
// 2^-150), d is a power of two that keeps c at 2^-100 or, past d's own range, as
// near as it gets: x c then is an ordinary number wherever x c d is not zero.
struct Factor { float c, d; };
__device__ __forceinline__ Factor factor_of(double ratio) {
  if (ratio > 1.0) return {1.0f, 1.0f};
  if (!(ratio > 0.0 && ratio < 0x1p-126)) return {(float)ratio, 1.0f};   // NaN and 0 among them
  const int e = max(__builtin_amdgcn_frexp_exp(ratio) + 100, -149);
  return {(float)ldexp(ratio, -e), ldexpf(1.0f, e)};
}

// c is 1 exactly, and x its own result, where norm + eps <= max_norm (and where
// the ratio rounds to 1: 2^-25 below it); a NaN norm makes c, and so every
// gradient, NaN.  in may be out.  Everything passes
// here once: past the caches (2.1 GB of norm, read and write 516 us, 564 through
// them; 134 MB of gradients 64 and 66; what then reads the gradients loses 1% at
// most).  The norm's pass keeps its loads in them for this one: nontemporal there
// too, 67 MB of gradients take 70 us in place of 63.
__global__ void __launch_bounds__(GN_THREADS)
clip_kernel(const Tensors t, const double* partials, int parts, float max_norm, float eps,
            float* __restrict__ norm) {
  __shared__ double s[GN_THREADS / 64];
  const double nv = sqrt(sum_of(partials, parts, s));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)nv;
  const double ratio = (double)max_norm / (nv + (double)eps);
  const Factor f = factor_of(ratio);
  const float c = f.c, d = f.d;
  for (uint32_t ch = blockIdx.x; ch < t.chunks; ch += gridDim.x) {
    const int i = tensor_of(t, ch);
    if (c == 1.0f && t.in[i] == t.out[i]) continue;   // nothing to change
    const int64_t at = (int64_t)(ch - t.first[i]) * GN_CHUNK;
    const int n = (int)(t.numel[i] - at < GN_CHUNK ? t.numel[i] - at : GN_CHUNK);
    int done = 0;
    if ((t.f32[i >> 5] >> (i & 31)) & 1u) {
      const float* p = static_cast<const float*>(t.in[i]) + at;
      float* o = static_cast<float*>(t.out[i]) + at;
      if (aligned16(p) && aligned16(o)) {
        done = n & ~3;
#pragma unroll 4
        for (int e = threadIdx.x * 4; e < done; e += GN_THREADS * 4) {
          v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p + e));
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * c * d);
          __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(o + e));
        }
      }
      for (int e = done + threadIdx.x; e < n; e += GN_THREADS) o[e] = p[e] * c * d;
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(t.in[i]) + at;
      uint16_t* o = static_cast<uint16_t*>(t.out[i]) + at;
      if (aligned16(p) && aligned16(o)) {
        done = n & ~7;
#pragma unroll 4
        for (int e = threadIdx.x * 8; e < done; e += GN_THREADS * 8) {
          v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p + e));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const v2f x = {__uint_as_float(v[j] << 16) * c * d, __uint_as_float(v[j] & 0xffff0000u) * c * d};
            v[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2bf));
          }
          __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(o + e));
        }
      }
      for (int e = done + threadIdx.x; e < n; e += GN_THREADS)
        o[e] = __builtin_bit_cast(uint16_t, (__bf16)(__uint_as_float((uint32_t)p[e] << 16) * c * d));
    }
  }
}

}  // namespace

int grad_norm_parts(const int64_t* numel, int n) {
  int64_t parts = 0;
  for (int i = 0; i < n; i += GN_TENSORS) {
    int64_t chunks = 0;
    for (int j = i; j < std::min(n, i + GN_TENSORS); ++j) chunks += (numel[j] + GN_CHUNK - 1) / GN_CHUNK;
    parts += std::min<int64_t>(chunks, GN_GRID);
  }
  return (int)parts;
}

hipError_t launch_clip_grads(const void* const* in, void* const* out, const int64_t* numel, const int* types, int n,
                             float max_norm, float eps, double* partials, float* norm, hipStream_t stream) {
  const int total = grad_norm_parts(numel, n);
  const bool clip = out != nullptr;
  // The norm inside the clipping kernel, once per workgroup, where there is one
  // launch of each: a launch less.  With more, the parts are too many for that.
  const bool fused = clip && n <= GN_TENSORS && total > 0;
  for (int pass = 0; pass < (clip ? 2 : 1); ++pass) {
    int at = 0;
    for (int i = 0; i < n; i += GN_TENSORS) {
      Tensors t{};
      int64_t chunks = 0;
      for (int j = i; j < std::min(n, i + GN_TENSORS); ++j) {
        if (numel[j] == 0) continue;
        t.in[t.n] = in[j];
        t.out[t.n] = clip ? out[j] : nullptr;
        t.numel[t.n] = numel[j];
        t.first[t.n] = (uint32_t)chunks;
        if (types[j] == 0) t.f32[t.n >> 5] |= 1u << (t.n & 31);
        chunks += (numel[j] + GN_CHUNK - 1) / GN_CHUNK;
        ++t.n;
      }
      if (chunks == 0) continue;
      t.chunks = (uint32_t)chunks;
      const int grid = (int)std::min<int64_t>(chunks, GN_GRID);
      if (pass == 0)
        hipLaunchKernelGGL(square_sum_kernel, dim3(grid), dim3(GN_THREADS), 0, stream, t, partials + at);
      else
        hipLaunchKernelGGL(clip_kernel, dim3(grid), dim3(GN_THREADS), 0, stream, t, partials + (fused ? 0 : total),
                           fused ? total : 1, max_norm, eps, fused ? norm : nullptr);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      at += grid;
    }
    if (pass == 0 && !fused) {
      hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(GN_THREADS), 0, stream, partials, total, norm);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace w4a8
