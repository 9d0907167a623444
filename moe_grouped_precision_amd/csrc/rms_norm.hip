// Root-mean-square norm with the residual's addition, output in bf16 and / or
// E4M3 with a scale per 128, and its gradient, gfx950.
//
//   h = bf16(x + r),  inv = (sum h^2 / K + eps)^(-1/2),  xh = h inv,  y = xh w
//   codes: per (row, 128 of y in fp32) s = amax / 448 (1 where amax < 2^-100),
//          code = E4M3(y * (1 / s))
//   gradient: g = dy w,  dh = inv (g - xh sum(g xh) / K) [+ dres],
//             dw = sum over the rows of dy xh
//
// A row lives in the registers of its threads (8 columns per 16-byte load) from
// the loads to the stores, so every input is read once; both sums of a row are
// taken in 64 bits, which hold the squares of any bf16 value (fp32 overflows
// from 2^64 on), and inv is applied in two factors, so that rows of the
// largest and the smallest values come out like any other.
//
// Bound by HBM: 16384 x 6144 with the residual, 805 MB, 136 us (5.9 TB/s; stores in
// the caches' way 141, 101 MB of output 74 in place of 58; what then reads the
// output takes within 2% of the same); the gradient of 16383 x 6144 with dres, 805
// MB, 145 and 5 for dw (5.5; in the caches' way 153, with a division by K for each
// sum 182).  64 rows to 8 bits: 4.1 us, a launch and a trip to memory.
#include "swiglu.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace w4a8 {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100
constexpr int NORM_WAVES = 16;       // most waves of a workgroup
constexpr int NORM_CHUNKS = 4;       // most chunks of 8 columns that a thread holds
constexpr int GRAD_WAVES = 8;        // of the gradient, whose threads hold three rows' chunks and dw

// 8 bf16 columns of a row.  VEC: 16-byte aligned and whole.  Otherwise a chunk
// may start at any 2 bytes and its last n < 8 columns are read one by one (what
// is past them counts as 0).
template <bool VEC>
__device__ __forceinline__ v4u load_chunk(const uint16_t* p, int n) {
  v4u a = {0, 0, 0, 0};
  if (VEC) {
    a = *reinterpret_cast<const v4u*>(p);
  } else if (n >= 8) {
    __builtin_memcpy(&a, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) a[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
  return a;
}
template <bool VEC>
__device__ __forceinline__ void store_chunk(uint16_t* p, v4u a, int n) {
  if (VEC) {
    __builtin_nontemporal_store(a, reinterpret_cast<v4u*>(p));
  } else if (n >= 8) {
    __builtin_memcpy(p, &a, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint16_t)(a[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void unpack(v4u a, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(a[i] << 16);
    f[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ v4u pack(const float (&f)[8]) {
  v4u a;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * i], f[2 * i + 1]}, v2bf));
  return a;
}

// 8 weights: bf16, fp32 or (null) ones.
template <bool VEC>
__device__ __forceinline__ void load_weights(const void* w, int f32, int k, int n, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.0f;
  } else if (!f32) {
    unpack(load_chunk<VEC>(static_cast<const uint16_t*>(w) + k, n), f);
  } else {
    const float* p = static_cast<const float*>(w) + k;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = VEC || i < n ? p[i] : 0.0f;
  }
}

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum over the 64 lanes, in each of them (the same bits in all).
__device__ __forceinline__ double wave_sum(double v) {
  v = add_dpp<0x128>(v);   // row_ror 8, 4, 2, 1
  v = add_dpp<0x124>(v);
  v = add_dpp<0x122>(v);
  v = add_dpp<0x121>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
  return fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true)));
}

// v^(-1/2) as c1 * c2, c1 a power of two and both inside fp32's normal range
// for every v of bf16 rows (2^-266 to 2^256): (x c1) c2 neither overflows nor
// loses bits where x v^(-1/2) is an ordinary number.  v = 0 gives infinity
// (rows of zeros with eps = 0 are NaN), infinity 0, NaN NaN.
struct Inv { float c1, c2; };
__device__ __forceinline__ Inv inv_sqrt(double v) {
  if (!(v > 0.0) || v > 1.7e308) {
    const float one = 1.0f;
    return {one, v == 0.0 ? __builtin_inff() : v > 0.0 ? 0.0f : __builtin_nanf("")};
  }
  int e = __builtin_amdgcn_frexp_exp(v);
  double m = __builtin_amdgcn_frexp_mant(v);   // [1/2, 1)
  if (e & 1) {
    m *= 2.0;
    e -= 1;
  }
  const float f = (float)m;
  float r = __builtin_amdgcn_rsqf(f);
  r = fmaf(r * 0.5f, fmaf(-f * r, r, 1.0f), r);   // one Newton step
  const int p = -e / 2, p1 = p >> 1;
  return {ldexpf(1.0f, p1), ldexpf(r, p - p1)};
}

// Sum of a row's N values over its waves: in registers for one wave, through
// LDS otherwise.  Two sets of places in turn, so that one barrier per row does
// (a wave is at most one row ahead of another).
template <int N>
__device__ __forceinline__ void row_sum(double (&v)[N], int waves, double (*s)[N][NORM_WAVES], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s[turn][i][threadIdx.x >> 6] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    double a = 0.0;
    for (int w = 0; w < waves; ++w) a += s[turn][i][w];
    v[i] = a;
  }
  turn ^= 1;
}

struct RowPlace { int tid, threads, waves; int64_t t; bool live; };
// The threads of a row: all of the workgroup's, or with `rows_per` > 1 those of
// one wave (no barrier, and a wave without a row leaves).
__device__ __forceinline__ RowPlace place_of(int rows_per, int64_t first, int64_t T) {
  if (rows_per == 1) return {(int)threadIdx.x, (int)blockDim.x, (int)(blockDim.x >> 6), first, first < T};
  const int64_t t = first * rows_per + (threadIdx.x >> 6);
  return {(int)(threadIdx.x & 63), 64, 1, t, t < T};
}

// One lane's 8 columns of y to E4M3 with the scale of its 16 lanes' 128.  No
// clip: |y / s| stays under 448 (1 + 2^-22), which rounds to 448; NaN keeps a
// NaN code, an infinity makes its group's scale infinite and the group NaN.
__device__ __forceinline__ void quant_chunk(const float (&y)[8], uint8_t* codes, float* scale, bool write_scale) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
  m = max_dpp<0x128>(m);
  m = max_dpp<0x124>(m);
  m = max_dpp<0x122>(m);
  m = max_dpp<0x121>(m);
  const float s = m < kScaleFloor ? 1.0f : __fdiv_rn(m, 448.0f);
  const float inv = __fdiv_rn(1.0f, s);
  v2u c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] * inv, y[4 * i + 1] * inv, 0, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] * inv, y[4 * i + 3] * inv, q, true);
    c[i] = (uint32_t)q;
  }
  *reinterpret_cast<v2u*>(codes) = c;
  if (write_scale) *scale = s;
}

// x and res may be the buffers of y and h: every chunk is read before it is
// written, by the same thread (hence no __restrict__ on them).
template <int NCH, bool VEC>
__global__ void __launch_bounds__(64 * NORM_WAVES)
rms_norm_kernel(NormArgs a, int rows_per, int64_t row0) {
  __shared__ double sums[2][1][NORM_WAVES];
  // M-major scales: consecutive rows on one XCD, whose L2 then joins their
  // 4-byte scales to lines
  const uint32_t nb = gridDim.x;
  const uint32_t b = a.A && a.layout && !(nb & 7) ? (blockIdx.x & 7) * (nb >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  const RowPlace r = place_of(rows_per, b, a.T - row0);
  if (!r.live) return;
  const size_t t = (size_t)(row0 + r.t), base = t * a.K;
  const double ik = 1.0 / a.K;
  float f[NCH][8];
  double ss[1] = {0.0};
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int k = (r.tid + j * r.threads) * 8, n = a.K - k;
    v4u v = {0, 0, 0, 0};
    if (n > 0) {
      v = load_chunk<VEC>(a.x + base + k, n);
      if (a.res) {
        float g[8];
        unpack(v, f[j]);
        unpack(load_chunk<VEC>(a.res + base + k, n), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[j][i] += g[i];
        v = pack(f[j]);
      }
    }
    unpack(v, f[j]);
    if (n > 0 && a.h) store_chunk<VEC>(a.h + base + k, v, n);
  }
#pragma unroll
  for (int j = 0; j < NCH; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] = fma((double)f[j][i], (double)f[j][i], ss[0]);
  int turn = 0;
  row_sum<1>(ss, r.waves, sums, turn);
  const Inv c = inv_sqrt(ss[0] * ik + (double)a.eps);
  const int G = a.K >> 7;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int k = (r.tid + j * r.threads) * 8, n = a.K - k;
    if (n <= 0) break;
    float w[8], y[8];
    load_weights<VEC>(a.w, a.w_f32, k, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = f[j][i] * c.c1 * c.c2 * w[i];
    if (a.y) store_chunk<VEC>(a.y + base + k, pack(y), n);
    if (a.A) {
      const int g = k >> 7;
      quant_chunk(y, a.A + base + k, a.SA + (a.layout ? (size_t)g * a.T + t : t * G + g), (threadIdx.x & 15) == 0);
    }
  }
}

// Rows past what the registers of a workgroup hold (K > 32768): the same in two
// passes over the row.
template <bool VEC>
__global__ void __launch_bounds__(64 * NORM_WAVES)
rms_norm_long_kernel(NormArgs a, int64_t row0) {
  __shared__ double sums[2][1][NORM_WAVES];
  const size_t t = (size_t)(row0 + blockIdx.x), base = t * a.K;
  const int G = a.K >> 7;
  const double ik = 1.0 / a.K;
  double ss[1] = {0.0};
  float f[8], g[8];
  for (int k = threadIdx.x * 8; k < a.K; k += blockDim.x * 8) {
    const int n = a.K - k;
    v4u v = load_chunk<VEC>(a.x + base + k, n);
    unpack(v, f);
    if (a.res) {
      unpack(load_chunk<VEC>(a.res + base + k, n), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += g[i];
      v = pack(f);
      unpack(v, f);
    }
    if (a.h) store_chunk<VEC>(a.h + base + k, v, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] = fma((double)f[i], (double)f[i], ss[0]);
  }
  int turn = 0;
  row_sum<1>(ss, blockDim.x >> 6, sums, turn);
  const Inv c = inv_sqrt(ss[0] * ik + (double)a.eps);
  for (int k = threadIdx.x * 8; k < a.K; k += blockDim.x * 8) {
    const int n = a.K - k;
    float w[8], y[8];
    // h from where this thread wrote it: x or res may be gone under it
    unpack(load_chunk<VEC>((a.h ? a.h : a.x) + base + k, n), f);
    if (a.res && !a.h) {
      unpack(load_chunk<VEC>(a.res + base + k, n), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += g[i];
      unpack(pack(f), f);
    }
    load_weights<VEC>(a.w, a.w_f32, k, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = f[i] * c.c1 * c.c2 * w[i];
    if (a.y) store_chunk<VEC>(a.y + base + k, pack(y), n);
    if (a.A) {
      const int gr = k >> 7;
      quant_chunk(y, a.A + base + k, a.SA + (a.layout ? (size_t)gr * a.T + t : t * G + gr), (threadIdx.x & 15) == 0);
    }
  }
}

// The gradient: workgroup b takes rows b, b + gridDim.x, ... and keeps its part
// of dw in registers, an fp32 sum of ceil(T / 512) products (in 64 bits it would
// take twice the registers), written to partials[b][K] at the end.
template <int NCH, bool VEC>
__global__ void __launch_bounds__(64 * GRAD_WAVES)
rms_norm_backward_kernel(NormGradArgs a) {
  __shared__ double sums[2][2][NORM_WAVES];
  const int waves = blockDim.x >> 6;
  const double ik = 1.0 / a.K;
  float w[NCH][8], dw[NCH][8];
  v4u hv[NCH], dv[NCH], rv[NCH];
  auto load_row = [&](int64_t t) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int k = (threadIdx.x + j * blockDim.x) * 8, n = a.K - k;
      const size_t at = (size_t)t * a.K + k;
      hv[j] = dv[j] = rv[j] = (v4u){0, 0, 0, 0};
      if (n > 0) {
        hv[j] = load_chunk<VEC>(a.h + at, n);
        dv[j] = load_chunk<VEC>(a.dy + at, n);
        if (a.dres) rv[j] = load_chunk<VEC>(a.dres + at, n);
      }
    }
  };
  load_row(blockIdx.x);
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int k = (threadIdx.x + j * blockDim.x) * 8, n = a.K - k;
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = w[j][i] = 0.f;
    if (n > 0) load_weights<VEC>(a.w, a.w_f32, k, n, w[j]);
  }
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    v4u h0[NCH], d0[NCH], r0[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      h0[j] = hv[j];
      d0[j] = dv[j];
      r0[j] = rv[j];
    }
    if (t + gridDim.x < a.T) load_row(t + gridDim.x);   // in flight during this row
    double s[2] = {0.0, 0.0};   // sum h^2, sum g h
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      float f[8], d[8];
      unpack(h0[j], f);
      unpack(d0[j], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] = fma((double)f[i], (double)f[i], s[0]);
        s[1] = fma((double)(d[i] * w[j][i]), (double)f[i], s[1]);
      }
    }
    row_sum<2>(s, waves, sums, turn);
    const Inv c = inv_sqrt(s[0] * ik + (double)a.eps);
    // sum(g xh) / K
    const float m = (float)(s[1] * (double)c.c1 * (double)c.c2 * ik);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int k = (threadIdx.x + j * blockDim.x) * 8, n = a.K - k;
      if (n <= 0) break;
      float f[8], d[8], r[8], o[8];
      unpack(h0[j], f);
      unpack(d0[j], d);
      unpack(r0[j], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = f[i] * c.c1 * c.c2;
        dw[j][i] = fmaf(d[i], xh, dw[j][i]);
        o[i] = fmaf(-xh, m, d[i] * w[j][i]) * c.c1 * c.c2 + r[i];
      }
      store_chunk<VEC>(a.dx + (size_t)t * a.K + k, pack(o), n);
    }
  }
  float* part = a.partials + (size_t)blockIdx.x * a.K;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const int k = (threadIdx.x + j * blockDim.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < a.K) part[k + i] = dw[j][i];
  }
}

// Rows past a workgroup's registers: two passes over the row, dw's part kept in
// partials (each place by one thread).
template <bool VEC>
__global__ void __launch_bounds__(64 * NORM_WAVES)
rms_norm_backward_long_kernel(NormGradArgs a) {
  __shared__ double sums[2][2][NORM_WAVES];
  float* part = a.partials + (size_t)blockIdx.x * a.K;
  const double ik = 1.0 / a.K;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t base = (size_t)t * a.K;
    double s[2] = {0.0, 0.0};
    for (int k = threadIdx.x * 8; k < a.K; k += blockDim.x * 8) {
      const int n = a.K - k;
      float f[8], d[8], w[8];
      unpack(load_chunk<VEC>(a.h + base + k, n), f);
      unpack(load_chunk<VEC>(a.dy + base + k, n), d);
      load_weights<VEC>(a.w, a.w_f32, k, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[0] = fma((double)f[i], (double)f[i], s[0]);
        s[1] = fma((double)(d[i] * w[i]), (double)f[i], s[1]);
      }
    }
    row_sum<2>(s, blockDim.x >> 6, sums, turn);
    const Inv c = inv_sqrt(s[0] * ik + (double)a.eps);
    const float m = (float)(s[1] * (double)c.c1 * (double)c.c2 * ik);
    for (int k = threadIdx.x * 8; k < a.K; k += blockDim.x * 8) {
      const int n = a.K - k;
      float f[8], d[8], w[8], r[8] = {0, 0, 0, 0, 0, 0, 0, 0}, o[8];
      unpack(load_chunk<VEC>(a.h + base + k, n), f);
      unpack(load_chunk<VEC>(a.dy + base + k, n), d);
      if (a.dres) unpack(load_chunk<VEC>(a.dres + base + k, n), r);
      load_weights<VEC>(a.w, a.w_f32, k, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = f[i] * c.c1 * c.c2;
        if (k + i < a.K) part[k + i] = fmaf(d[i], xh, t == blockIdx.x ? 0.0f : part[k + i]);
        o[i] = fmaf(-xh, m, d[i] * w[i]) * c.c1 * c.c2 + r[i];
      }
      store_chunk<VEC>(a.dx + base + k, pack(o), n);
    }
  }
}

// dw[k] = sum over the workgroups' parts, 32 columns and 32 runs of parts per
// workgroup, in 64 bits and a fixed order.
__global__ void __launch_bounds__(1024)
norm_weight_sum_kernel(const float* __restrict__ partials, int parts, int K, float* __restrict__ dw) {
  __shared__ double s[32][33];
  const int c = threadIdx.x & 31, k = blockIdx.x * 32 + c, run = threadIdx.x >> 5;
  double v = 0.0;
  if (k < K) {
    const float* p = partials + (size_t)run * K + k;
#pragma unroll 8
    for (int i = run; i < parts; i += 32, p += (size_t)32 * K) v += (double)*p;
  }
  s[run][c] = v;
  __syncthreads();
  if (run == 0 && k < K) {
    for (int i = 1; i < 32; ++i) v += s[i][c];
    dw[k] = (float)v;
  }
}

bool vec_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int norm_backward_parts(int T) { return std::min(T, NORM_PARTS); }

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
  const int chunks = (a.K + 7) / 8;
  const bool vec = a.K % 8 == 0 && vec_ok(a.x) && vec_ok(a.res) && vec_ok(a.y) && vec_ok(a.h) && vec_ok(a.w);
  const int most = 64 * NORM_WAVES;
  if (chunks > most * NORM_CHUNKS) {
    return in_launches(a.T, most, [&](int64_t t, int64_t n) {
      if (vec) hipLaunchKernelGGL(rms_norm_long_kernel<true>, dim3((unsigned)n), dim3(most), 0, stream, a, t);
      else hipLaunchKernelGGL(rms_norm_long_kernel<false>, dim3((unsigned)n), dim3(most), 0, stream, a, t);
    });
  }
  int nch = a.T <= 1024 ? 1 : 2;
  while ((chunks + nch - 1) / nch > most) nch *= 2;
  const int threads = ((chunks + nch - 1) / nch + 63) / 64 * 64;
  const int rows_per = threads == 64 ? 4 : 1, block = threads * rows_per;
  return in_launches(((int64_t)a.T + rows_per - 1) / rows_per, block, [&](int64_t b, int64_t n) {
    const dim3 grid((unsigned)n), blk(block);
    const int64_t t = b * rows_per;
#define W4A8_NORM(N)                                                                              \
  if (vec) hipLaunchKernelGGL((rms_norm_kernel<N, true>), grid, blk, 0, stream, a, rows_per, t);  \
  else hipLaunchKernelGGL((rms_norm_kernel<N, false>), grid, blk, 0, stream, a, rows_per, t)
    if (nch == 1) { W4A8_NORM(1); }
    else if (nch == 2) { W4A8_NORM(2); }
    else { W4A8_NORM(4); }
#undef W4A8_NORM
  });
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t stream) {
  const int chunks = (a.K + 7) / 8, parts = norm_backward_parts(a.T);
  const bool vec = a.K % 8 == 0 && vec_ok(a.h) && vec_ok(a.dy) && vec_ok(a.dres) && vec_ok(a.dx) && vec_ok(a.w);
  if (parts > 0) {
    const int most = 64 * GRAD_WAVES;
    int nch = chunks <= 256 ? 1 : 2;
    if (chunks > most * nch) nch = 4;
    const int threads = std::min(most, ((chunks + nch - 1) / nch + 63) / 64 * 64);
    const dim3 grid(parts), blk(threads);
#define W4A8_NORM(N)                                                                        \
  if (vec) hipLaunchKernelGGL((rms_norm_backward_kernel<N, true>), grid, blk, 0, stream, a); \
  else hipLaunchKernelGGL((rms_norm_backward_kernel<N, false>), grid, blk, 0, stream, a)
    if (chunks > most * NORM_CHUNKS) {
      if (vec) hipLaunchKernelGGL(rms_norm_backward_long_kernel<true>, grid, dim3(64 * NORM_WAVES), 0, stream, a);
      else hipLaunchKernelGGL(rms_norm_backward_long_kernel<false>, grid, dim3(64 * NORM_WAVES), 0, stream, a);
    } else if (nch == 1) { W4A8_NORM(1); }
    else if (nch == 2) { W4A8_NORM(2); }
    else { W4A8_NORM(4); }
#undef W4A8_NORM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw)
    hipLaunchKernelGGL(norm_weight_sum_kernel, dim3((a.K + 31) / 32), dim3(1024), 0, stream, a.partials, parts, a.K, a.dw);
  return hipGetLastError();
}

}  // namespace w4a8
