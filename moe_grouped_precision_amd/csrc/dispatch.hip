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
// Streams bound by HBM, 8 columns (16 bytes) per lane; rows that are not
// 16-byte multiples, or start elsewhere, go 1 column per lane.
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
  __device__ __forceinline__ void load_once(const uint16_t* p) {
    v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<v4u*>(p) = v; }
  __device__ __forceinline__ void store_once(uint16_t* p) const {
    __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(p));
  }
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
  __device__ __forceinline__ void load_once(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = v; }
  __device__ __forceinline__ void store_once(uint16_t* p) const { *p = v; }
  __device__ __forceinline__ void floats(float (&f)[1]) const { f[0] = __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ void from(const float (&f)[1]) { v = __builtin_bit_cast(uint16_t, (__bf16)f[0]); }
};

// A token's columns stay in registers while its rows are written one after
// the other, two chunks per lane and up to 512 lanes.  89% of the bytes of a
// top-8 dispatch are writes to rows all over A, and these bound it: 16384 x
// 6144 takes 345 us, 5.2 TB/s (a plain fill of A: 233 us); 361 us with the
// loads nontemporal, 365 with the stores, 354 with six chunks per lane, 450
// when every row of A is written by a workgroup of its own in row order.
constexpr int D_LANES = 512, D_CHUNKS = 2;
template <int W>
__global__ void __launch_bounds__(D_LANES)
dispatch_kernel(const uint16_t* __restrict__ x, int K, const int32_t* __restrict__ row_of_slot, int top_k, int R,
                uint16_t* __restrict__ A) {
  const size_t t = blockIdx.x;
  const int32_t* rs = row_of_slot + t * top_k;
  const int step = blockDim.x * W;
  for (int c0 = threadIdx.x * W; c0 < K; c0 += step * D_CHUNKS) {
    Cols<W> v[D_CHUNKS];
#pragma unroll
    for (int i = 0; i < D_CHUNKS; ++i) {
      const int c = c0 + i * step;
      if (c < K) v[i].load(x + t * K + c);
    }
    for (int j = 0; j < top_k; ++j) {
      const int r = rs[j];
      if (r < 0 || r >= R) continue;
#pragma unroll
      for (int i = 0; i < D_CHUNKS; ++i) {
        const int c = c0 + i * step;
        if (c < K) v[i].store(A + (size_t)r * K + c);
      }
    }
  }
}

// One workgroup per token and 256 chunks, so that the last round of
// workgroups is short (1151 tokens x 6144, top-8: 22.8 us, 5.3 TB/s; 25.1
// with a workgroup per token).  Nontemporal loads: 25.5 without.
constexpr int B_LANES = 256;
template <int W>
__global__ void __launch_bounds__(B_LANES)
dispatch_backward_kernel(const uint16_t* __restrict__ dA, int R, int K, const int32_t* __restrict__ row_of_slot,
                         int top_k, uint16_t* __restrict__ dx, int segments) {
  const size_t t = blockIdx.x / (unsigned)segments;
  const int32_t* rs = row_of_slot + t * top_k;
  for (int c = ((int)(blockIdx.x - t * segments) * B_LANES + (int)threadIdx.x) * W; c < K; c += segments * B_LANES * W) {
    float acc[W] = {};
    // eight slots' loads in flight at once, then their terms in slot order
    for (int j0 = 0; j0 < top_k; j0 += 8) {
      Cols<W> v[8];
      bool ok[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = j0 + u < top_k ? rs[j0 + u] : -1;
        ok[u] = r >= 0 && r < R;
        if (ok[u]) v[u].load_once(dA + (size_t)r * K + c);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (!ok[u]) continue;
        float f[W];
        v[u].floats(f);
#pragma unroll
        for (int i = 0; i < W; ++i) acc[i] += f[i];
      }
    }
    Cols<W> o;
    o.from(acc);
    o.store(dx + t * K + c);
  }
}

// Two waves per slot, each with six chunks of C and of dout in flight: 1152 x
// 6144, top-8 45.3 us; one wave and one chunk 53.0, one wave and six 46.1,
// four waves and three 49.0.  Workgroups go to the 8 XCDs in turn, so four
// neighbouring ones (8 slots: mostly one token's) are dealt to the same XCD, whose
// L2 then serves dout's row to all of them (44.7 us, 5.3 TB/s).
constexpr int C_SPLIT = 2, C_CHUNKS = 6, C_WAVES = 4;
template <int W>
__global__ void __launch_bounds__(64 * C_WAVES)
combine_backward_kernel(const uint16_t* __restrict__ C, const uint16_t* __restrict__ dout, int R, int N,
                        const int32_t* __restrict__ row_of_slot, const float* __restrict__ weights, int64_t first,
                        int64_t slots, int top_k, uint16_t* __restrict__ dC, float* __restrict__ dweights) {
  __shared__ float part[C_WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t b = (blockIdx.x & ~31u) | (blockIdx.x & 7u) << 2 | (blockIdx.x >> 3 & 3u);
  const int64_t s = first + (int64_t)b * (C_WAVES / C_SPLIT) + wave / C_SPLIT;
  const int r = s < slots ? row_of_slot[s] : -1;
  float dot = 0.f;
  if (r >= 0 && r < R) {
    const float w = weights[s];
    const uint16_t* d = dout + (size_t)((uint32_t)s / (uint32_t)top_k) * N;
    const uint16_t* c = C + (size_t)r * N;
    uint16_t* o = dC + (size_t)r * N;
    constexpr int STEP = 64 * C_SPLIT * W;
    for (int i0 = ((wave % C_SPLIT) * 64 + lane) * W; i0 < N; i0 += STEP * C_CHUNKS) {
      Cols<W> a[C_CHUNKS], b[C_CHUNKS];
#pragma unroll
      for (int u = 0; u < C_CHUNKS; ++u)
        if (i0 + u * STEP < N) {
          a[u].load_once(c + i0 + u * STEP);
          b[u].load(d + i0 + u * STEP);
        }
#pragma unroll
      for (int u = 0; u < C_CHUNKS; ++u)
        if (i0 + u * STEP < N) {
          float fa[W], fb[W];
          a[u].floats(fa);
          b[u].floats(fb);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            dot = fmaf(fa[i], fb[i], dot);
            fb[i] *= w;
          }
          Cols<W> q;
          q.from(fb);
          q.store_once(o + i0 + u * STEP);
        }
    }
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) dot += __shfl_xor(dot, i, 64);
  }
  if (lane == 0) part[wave] = dot;
  __syncthreads();
  if (lane == 0 && wave % C_SPLIT == 0 && s < slots) dweights[s] = part[wave] + part[wave + 1];
}

bool wide(int K, const void* a, const void* b, const void* c = nullptr) {
  return K % 8 == 0 && (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
}
int segments(int K, int W) { return (K + B_LANES * W - 1) / (B_LANES * W); }   // of a token

}  // namespace

hipError_t launch_dispatch(const uint16_t* x, int T, int K, const int32_t* row_of_slot, int top_k, int R, uint16_t* A,
                           hipStream_t stream) {
  const bool w = wide(K, x, A);
  const int n = (int)(((int64_t)K + (w ? 15 : 1)) / (w ? 16 : 2));   // lanes of two chunks
  const int lanes = n >= D_LANES ? D_LANES : (n + 63) & ~63;
  return in_launches(T, lanes, [&](int64_t t, int64_t tokens) {
    const dim3 grid((unsigned)tokens), block(lanes);
    if (w)
      hipLaunchKernelGGL(dispatch_kernel<8>, grid, block, 0, stream, x + t * K, K, row_of_slot + t * top_k, top_k, R, A);
    else
      hipLaunchKernelGGL(dispatch_kernel<1>, grid, block, 0, stream, x + t * K, K, row_of_slot + t * top_k, top_k, R, A);
  });
}

hipError_t launch_dispatch_backward(const uint16_t* dA, int R, int K, const int32_t* row_of_slot, int T, int top_k,
                                    uint16_t* dx, hipStream_t stream) {
  const bool w = wide(K, dA, dx);
  const int n = segments(K, w ? 8 : 1);
  return in_launches(T, (int64_t)n * B_LANES, [&](int64_t t, int64_t tokens) {
    const dim3 grid((unsigned)(tokens * n)), block(B_LANES);
    if (w)
      hipLaunchKernelGGL(dispatch_backward_kernel<8>, grid, block, 0, stream, dA, R, K, row_of_slot + t * top_k, top_k,
                         dx + t * K, n);
    else
      hipLaunchKernelGGL(dispatch_backward_kernel<1>, grid, block, 0, stream, dA, R, K, row_of_slot + t * top_k, top_k,
                         dx + t * K, n);
  });
}

hipError_t launch_combine_backward(const uint16_t* C, const uint16_t* dout, int R, int N, const int32_t* row_of_slot,
                                   const float* weights, int T, int top_k, uint16_t* dC, float* dweights,
                                   hipStream_t stream) {
  const int64_t slots = (int64_t)T * top_k;
  constexpr int per_wg = C_WAVES / C_SPLIT;
  // launches of a multiple of 64 slots: whole sets of 32 workgroups (see b)
  return in_launches(slots, 64 * C_SPLIT, [&](int64_t s, int64_t n) {
    const dim3 grid((unsigned)((n + per_wg * 32 - 1) / (per_wg * 32) * 32)), block(64 * C_WAVES);
    if (wide(N, C, dout, dC))
      hipLaunchKernelGGL(combine_backward_kernel<8>, grid, block, 0, stream, C, dout, R, N, row_of_slot, weights, s,
                         slots, top_k, dC, dweights);
    else
      hipLaunchKernelGGL(combine_backward_kernel<1>, grid, block, 0, stream, C, dout, R, N, row_of_slot, weights, s,
                         slots, top_k, dC, dweights);
  });
}

}  // namespace w4a8
