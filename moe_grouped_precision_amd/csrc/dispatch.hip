// Tokens to the experts' rows, and the gradients of both moves, gfx950.
//
//   dispatch           A[row(t, j), :] = x[t, :]
//   its gradient       dx[t, :] = sum_j dA[row(t, j), :]
//   combine's gradient dC[row(t, j), :] = w[t, j] dout[t, :]
//                      dw[t, j] = <C[row(t, j), :], dout[t, :]>
// (combine, out[t, :] = sum_j w[t, j] C[row(t, j), :], is combine.hip's.)
// Sums run in fp32, one rounding to bf16 at the end; no atomics, so the
// results are the same on every call.
//
// Streams bound by HBM: one workgroup per token, 8 columns (one 16-byte
// load) per lane; rows that are not 16-byte multiples go 1 column per lane.
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

namespace w4a8 {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// W columns of one row: 8 as four dwords, 1 as a half word.
template <int W>
struct Cols;
template <>
struct Cols<8> {
  v4u v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const v4u*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<v4u*>(p) = v; }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void from(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * i], f[2 * i + 1]}, v2bf));
  }
};
template <>
struct Cols<1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = v; }
  __device__ __forceinline__ void floats(float (&f)[1]) const { f[0] = __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ void from(const float (&f)[1]) { v = __builtin_bit_cast(uint16_t, (__bf16)f[0]); }
};

template <int W>
__global__ void __launch_bounds__(512)
dispatch_kernel(const uint16_t* __restrict__ x, int K, const int32_t* __restrict__ row_of_slot, int top_k, int R,
                uint16_t* __restrict__ A) {
  const size_t t = blockIdx.x;
  const int32_t* rs = row_of_slot + t * top_k;
  for (int c = threadIdx.x * W; c < K; c += blockDim.x * W) {
    Cols<W> v;
    v.load(x + t * K + c);
    for (int j = 0; j < top_k; ++j) {
      const int r = rs[j];
      if (r >= 0 && r < R) v.store(A + (size_t)r * K + c);
    }
  }
}

template <int W>
__global__ void __launch_bounds__(512)
dispatch_backward_kernel(const uint16_t* __restrict__ dA, int R, int K, const int32_t* __restrict__ row_of_slot,
                         int top_k, uint16_t* __restrict__ dx) {
  const size_t t = blockIdx.x;
  const int32_t* rs = row_of_slot + t * top_k;
  for (int c = threadIdx.x * W; c < K; c += blockDim.x * W) {
    float acc[W] = {};
    for (int j = 0; j < top_k; ++j) {
      const int r = rs[j];
      if (r < 0 || r >= R) continue;
      Cols<W> v;
      v.load(dA + (size_t)r * K + c);
      float f[W];
      v.floats(f);
#pragma unroll
      for (int i = 0; i < W; ++i) acc[i] += f[i];
    }
    Cols<W> o;
    o.from(acc);
    o.store(dx + t * K + c);
  }
}

// One wave per slot.
template <int W>
__global__ void __launch_bounds__(256)
combine_backward_kernel(const uint16_t* __restrict__ C, const uint16_t* __restrict__ dout, int R, int N,
                        const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights, int slots,
                        int top_k, uint16_t* __restrict__ dC, float* __restrict__ dweights) {
  const int lane = threadIdx.x & 63;
  const int64_t s = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (s >= slots) return;
  const int r = row_of_slot[s];
  float dot = 0.f;
  if (r >= 0 && r < R) {
    const float w = weights[s];
    const uint16_t* d = dout + (size_t)(s / top_k) * N;
    for (int c = lane * W; c < N; c += 64 * W) {
      Cols<W> a, b, o;
      a.load(C + (size_t)r * N + c);
      b.load(d + c);
      float fa[W], fb[W];
      a.floats(fa);
      b.floats(fb);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        dot = fmaf(fa[i], fb[i], dot);
        fb[i] *= w;
      }
      o.from(fb);
      o.store(dC + (size_t)r * N + c);
    }
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) dot += __shfl_xor(dot, i, 64);
  }
  if (lane == 0) dweights[s] = dot;
}

bool wide(int K, const void* a, const void* b, const void* c = nullptr) {
  return K % 8 == 0 && (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
}
int lanes(int K, int W) {  // whole waves, at most 512 lanes
  const int n = (K + W - 1) / W;
  return n >= 512 ? 512 : (n + 63) & ~63;
}

}  // namespace

hipError_t launch_dispatch(const uint16_t* x, int T, int K, const int32_t* row_of_slot, int top_k, int R, uint16_t* A,
                           hipStream_t stream) {
  if (wide(K, x, A))
    hipLaunchKernelGGL(dispatch_kernel<8>, dim3(T), dim3(lanes(K, 8)), 0, stream, x, K, row_of_slot, top_k, R, A);
  else
    hipLaunchKernelGGL(dispatch_kernel<1>, dim3(T), dim3(lanes(K, 1)), 0, stream, x, K, row_of_slot, top_k, R, A);
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const uint16_t* dA, int R, int K, const int32_t* row_of_slot, int T, int top_k,
                                    uint16_t* dx, hipStream_t stream) {
  if (wide(K, dA, dx))
    hipLaunchKernelGGL(dispatch_backward_kernel<8>, dim3(T), dim3(lanes(K, 8)), 0, stream, dA, R, K, row_of_slot,
                       top_k, dx);
  else
    hipLaunchKernelGGL(dispatch_backward_kernel<1>, dim3(T), dim3(lanes(K, 1)), 0, stream, dA, R, K, row_of_slot,
                       top_k, dx);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const uint16_t* C, const uint16_t* dout, int R, int N, const int32_t* row_of_slot,
                                   const float* weights, int T, int top_k, uint16_t* dC, float* dweights,
                                   hipStream_t stream) {
  const int slots = T * top_k;
  const dim3 grid((slots + 3) / 4);
  if (wide(N, C, dout, dC))
    hipLaunchKernelGGL(combine_backward_kernel<8>, grid, dim3(256), 0, stream, C, dout, R, N, row_of_slot, weights,
                       slots, top_k, dC, dweights);
  else
    hipLaunchKernelGGL(combine_backward_kernel<1>, grid, dim3(256), 0, stream, C, dout, R, N, row_of_slot, weights,
                       slots, top_k, dC, dweights);
  return hipGetLastError();
}

}  // namespace w4a8
