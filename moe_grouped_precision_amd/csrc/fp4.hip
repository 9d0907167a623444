// bf16 to 4-bit floating point with group scales and back, gfx950.
//
//   MXFP4 (32 along K): e = floor(log2 amax) - 2, scale 2^e as an E8M0 code (1 for a
//     group of zeros), code = E2M1 of x / 2^e
//   NVFP4 (16 along K): gs = amax of the expert / (6 * 448) in fp32 (1 for zeros),
//     s = E4M3(amax of the group / (6 gs)), code = E2M1 of x / (s gs)
// All roundings to nearest, halves to even, past 6 to 6: the codes are those of
// the exact quotients.  MX divides by powers of two, which is exact.  NV's
// quotients meet the grids' midpoints exactly when x and the amax share their
// mantissas, and come as near as 2^-33 to them otherwise (x has 8 significant
// bits, s 4, gs 24, a midpoint 3): both are told apart exactly.
//
// Streams: a thread holds 16 columns, i.e. an NVFP4 group, two threads an MX
// group.  Bound by HBM, 264 M weights: the experts' amax 91 us (5.8 TB/s), NVFP4
// from it 120 (5.6), back 112 (6.0); MXFP4 111 (6.0), back 127 (5.3).  Tried: NVFP4's
// weights read the second time past the caches, 4% slower from 16 experts of 4096 x
// 4096 on; from the end, where the amax pass left off, 3%.
#include "swiglu.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace w4a8 {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int Q_THREADS = 256;
constexpr int AMAX_UNROLL = 4;
constexpr int64_t INFINITY_CACHE = 256 << 20;   // bytes
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

struct Cols { v4u lo, hi; };   // 16 bf16 columns
__device__ __forceinline__ Cols load16(const uint16_t* p) {
  const v4u* q = reinterpret_cast<const v4u*>(p);
  return {q[0], q[1]};
}
__device__ __forceinline__ float col(const Cols& c, int i) {
  const uint32_t w = i < 8 ? c.lo[i >> 1] : c.hi[(i - 8) >> 1];
  return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}
// The bits of max |x| of the 16 columns; infinity or NaN come out above 0x7f7f....
__device__ __forceinline__ uint32_t amax_bits(const Cols& c) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, max((c.lo[i] << 16) & 0x7fffffffu, c.lo[i] & 0x7fff0000u));
    m = max(m, max((c.hi[i] << 16) & 0x7fffffffu, c.hi[i] & 0x7fff0000u));
  }
  return m;
}
constexpr uint32_t INF_BITS = 0x7f800000u;

// The codes and the scale of half an MX group; the other half is in the
// neighbouring lane (lane ^ 1).  A group with an infinity or a NaN gets the NaN
// scale.
__device__ __forceinline__ v2u mx_codes(const Cols& c, uint8_t& scale) {
  uint32_t m = amax_bits(c);
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, true));   // quad_perm 1 0 3 2
  if (m >= INF_BITS) {
    scale = 0xff;
    return (v2u){0u, 0u};
  }
  int e = m ? __builtin_amdgcn_frexp_expf(__uint_as_float(m)) - 3 : 0;
  e = e < -127 ? -127 : e;   // 125 at most
  scale = (uint8_t)(e + 127);
  v2u q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0;
#define W4A8_FP4(B)                                                                                           \
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, ldexpf(col(c, 8 * h + 2 * B), -e),                          \
                                               ldexpf(col(c, 8 * h + 2 * B + 1), -e), 1.0f, B)
    W4A8_FP4(0);
    W4A8_FP4(1);
    W4A8_FP4(2);
    W4A8_FP4(3);
#undef W4A8_FP4
    q[h] = w;
  }
  return q;
}

// Rows of bf16 to MXFP4 in place order: unit i holds columns 16 i .. 16 i + 15
// of the whole array (K % 32 == 0, so a pair of units is a group).
__global__ void __launch_bounds__(Q_THREADS)
quant_mx_kernel(const uint16_t* __restrict__ x, int64_t unit0, int64_t units, uint8_t* __restrict__ B,
                uint8_t* __restrict__ SB) {
  const int64_t i = unit0 + (int64_t)blockIdx.x * Q_THREADS + threadIdx.x;
  if (i >= units) return;   // units is even: a pair of lanes leaves together
  uint8_t s;
  const v2u q = mx_codes(load16(x + i * 16), s);
  *reinterpret_cast<v2u*>(B + i * 8) = q;
  if (!(i & 1)) SB[i >> 1] = s;
}

// Tokens to the grouped rows of their slots: a workgroup per token.
__global__ void __launch_bounds__(Q_THREADS)
quant_gather_mx_kernel(const uint16_t* __restrict__ x, int K, const int32_t* __restrict__ row_of_slot, int top_k,
                       int R, uint8_t* __restrict__ A, uint8_t* __restrict__ SA) {
  const int64_t t = blockIdx.x;
  const int32_t* rs = row_of_slot + t * top_k;
  for (int u = threadIdx.x; u < K / 16; u += blockDim.x) {
    uint8_t s;
    const v2u q = mx_codes(load16(x + t * K + u * 16), s);
    for (int j = 0; j < top_k; ++j) {
      const int r = rs[j];
      if (r < 0 || r >= R) continue;   // a slot that names no row
      *reinterpret_cast<v2u*>(A + (size_t)r * (K / 2) + u * 8) = q;
      if (!(u & 1)) SA[(size_t)r * (K / 32) + (u >> 1)] = s;
    }
  }
}

__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* s) {
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) m = max(m, s[w]);
  return m;
}

// Largest finite |x| of a part of an expert, as bits: partials[e][part].
__global__ void __launch_bounds__(Q_THREADS)
expert_amax_kernel(const uint16_t* __restrict__ x, int64_t units, int parts, int64_t b0,
                   uint32_t* __restrict__ partials) {
  __shared__ uint32_t s[Q_THREADS / 64];
  const int64_t b = b0 + blockIdx.x, e = b / parts;
  const uint16_t* xe = x + e * units * 16;
  uint32_t m = 0;
  const int64_t step = (int64_t)parts * Q_THREADS;
  for (int64_t u = (b - e * parts) * Q_THREADS + threadIdx.x; u < units; u += AMAX_UNROLL * step) {
    Cols c[AMAX_UNROLL];
#pragma unroll
    for (int i = 0; i < AMAX_UNROLL; ++i) {   // what is past the end: the first again
      const int64_t at = u + i * step;
      c[i] = load16(xe + (at < units ? at : u) * 16);
    }
#pragma unroll
    for (int i = 0; i < AMAX_UNROLL; ++i) {
      uint32_t v = amax_bits(c[i]);
      if (v >= INF_BITS) {   // rare: again, without what is not finite
        v = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t a = __float_as_uint(col(c[i], k)) & 0x7fffffffu;
          v = max(v, a < INF_BITS ? a : 0u);
        }
      }
      m = max(m, v);
    }
  }
  m = block_max(m, s);
  if (threadIdx.x == 0) partials[b] = m;
}

// Which of two neighbours of a grid, codes k and k + 1 and values v[0] < v[1], the
// quotient a / t goes to, a and t positive: a against the midpoint times t.  The
// midpoint's product with what `scale` holds of t is exact (at most 7 bits), and the
// fma rounds only the difference, whose sign it keeps.
__device__ __forceinline__ uint32_t nearer(uint32_t k, v2f v, float scale, float t, float a) {
  const float over = fmaf((v[0] + v[1]) * 0.5f * scale, -t, a);
  return k + (over > 0.0f || (over == 0.0f && (k & 1)));
}

// Quotients are taken in fp32, within 2^-21 of the true ones, and rounded once
// with 2^-20 less and once with 2^-20 more of their size; only where the two differ
// does the exact quotient decide (in about one element of a thousand: x and the
// amax share their mantissas).  All in 64 bits: 250 us for 264 M weights; these
// alone by division in 64 bits: 153, by nearer(): 120.
__global__ void __launch_bounds__(Q_THREADS)
quant_nv_kernel(const uint16_t* __restrict__ x, int64_t units, int64_t per_expert, int64_t b0, int parts,
                const uint32_t* __restrict__ partials, uint8_t* __restrict__ B, uint8_t* __restrict__ SB,
                float* __restrict__ gs) {
  __shared__ uint32_t sm[Q_THREADS / 64];
  constexpr float LESS = 1.0f - 0x1p-20f, MORE = 1.0f + 0x1p-20f;
  const int64_t b = b0 + blockIdx.x, e = b / per_expert;
  const int64_t u = (b - e * per_expert) * Q_THREADS + threadIdx.x;
  const int64_t i = e * units + u;
  Cols c = {};
  if (u < units) c = load16(x + i * 16);
  uint32_t m = 0;
  for (int p = threadIdx.x; p < parts; p += Q_THREADS) m = max(m, partials[e * parts + p]);
  m = block_max(m, sm);
  // below 2^-100 a scale of the fp32 range would lose its bits: such experts count as zeros
  const float g = __uint_as_float(m) >= kScaleFloor ? __fdiv_rn(__uint_as_float(m), 2688.0f) : 1.0f;
  if (b == e * per_expert && threadIdx.x == 0) gs[e] = g;
  if (u >= units) return;
  const float ig = __fdiv_rn(1.0f, g);
  const uint32_t am = amax_bits(c);
  v2u q = {0u, 0u};
  uint32_t code = 0x7f;   // NaN: a group with an infinity or a NaN
  if (am < INF_BITS) {
    const float a = __uint_as_float(am), r = a * ig * (1.0f / 6.0f);
    code = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r * LESS, r * MORE, 0, false);
    if ((code & 0xff) != (code >> 8 & 0xff)) {
      code &= 0xff;   // the lower one
      code = nearer(code, __builtin_amdgcn_cvt_pk_f32_fp8((int)(code | (code + 1) << 8), false), 6.0f, g, a);
    }
    code &= 0xff;
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
    const float inv = s > 0.0f ? ig * __builtin_amdgcn_rcpf(s) : 0.0f;   // s = 0: codes 0, signs kept
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t lo = 0, hi = 0;
#define W4A8_FP4(P)                                                                                                \
  {                                                                                                                \
    const float v = col(c, 8 * h + 2 * P) * inv, w = col(c, 8 * h + 2 * P + 1) * inv;                              \
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v * LESS, w * LESS, 1.0f, P);                                \
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, v * MORE, w * MORE, 1.0f, P);                                \
  }
      W4A8_FP4(0)
      W4A8_FP4(1)
      W4A8_FP4(2)
      W4A8_FP4(3)
#undef W4A8_FP4
      const v4u cols = h ? c.hi : c.lo;
      for (uint32_t todo = lo ^ hi; todo;) {
        const int at = (__ffs((int)todo) - 1) & ~3, j = at >> 2;   // element j of the 8
        const uint32_t pair = j < 4 ? (j < 2 ? cols[0] : cols[1]) : (j < 6 ? cols[2] : cols[3]);
        const float xf = __uint_as_float(j & 1 ? pair & 0xffff0000u : pair << 16);
        const uint32_t k = lo >> at & 7;   // the lower one, its sign apart
        const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(k | (k + 1) << 4, 1.0f, 0);
        lo += (nearer(k, v, s, g, fabsf(xf)) - k) << at;
        todo &= ~(15u << at);
      }
      q[h] = lo;
    }
  }
  *reinterpret_cast<v2u*>(B + i * 8) = q;
  SB[i] = (uint8_t)code;
}

// Codes to bf16: a thread decodes 8 columns.  value = bf16((code * s) gs), code
// * s exact in fp32.  PAST: the output is larger than the Infinity Cache and goes
// round it.  From MXFP4, then with a product that reads the weights, us, through
// it | round it: 201 MB 37, 96 | 49, 114; 268 MB 67, 131 | 64, 129; 1074 MB 257,
// 456 | 253, 429.
template <bool NV, bool PAST>
__global__ void __launch_bounds__(Q_THREADS)
dequant_kernel(const uint8_t* __restrict__ B, const uint8_t* __restrict__ SB, const float* __restrict__ gs,
               int64_t units, int64_t per_expert, int64_t b0, uint16_t* __restrict__ out) {
  const int64_t b = b0 + blockIdx.x, e = b / per_expert;
  const int64_t u = (b - e * per_expert) * Q_THREADS + threadIdx.x;
  if (u >= units) return;
  const int64_t i = e * units + u;
  const uint32_t* p = reinterpret_cast<const uint32_t*>(B + i * 4);
  const uint32_t q = PAST ? __builtin_nontemporal_load(p) : *p;
  const float g = gs ? gs[e] : 1.0f;
  const uint32_t sc = SB[NV ? i >> 1 : i >> 2];
  const float s = NV ? __builtin_amdgcn_cvt_f32_fp8((int)sc, 0) : 1.0f;
  const int ex = (int)sc - 127;
  const bool nan = !NV && sc == 0xff;
  v4u o;
#define W4A8_DEQ(J)                                                                                   \
  {                                                                                                   \
    v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, J);                                     \
    v[0] = (NV ? v[0] * s : ldexpf(v[0], ex)) * g;                                                    \
    v[1] = (NV ? v[1] * s : ldexpf(v[1], ex)) * g;                                                    \
    if (nan) v[0] = v[1] = __builtin_nanf("");                                                        \
    o[J] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));                            \
  }
  W4A8_DEQ(0)
  W4A8_DEQ(1)
  W4A8_DEQ(2)
  W4A8_DEQ(3)
#undef W4A8_DEQ
  if (PAST) __builtin_nontemporal_store(o, reinterpret_cast<v4u*>(out + i * 8));
  else *reinterpret_cast<v4u*>(out + i * 8) = o;
}

// Parts of an expert's amax: enough workgroups for the chip over all experts,
// few enough for every quantising workgroup to read them.
int amax_parts(int E, int64_t units) {
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(256, 2048 / E));
  return (int)std::min<int64_t>(most, (units + Q_THREADS - 1) / Q_THREADS);
}

}  // namespace

size_t quant_fp4_workspace(bool nv, int E, int N, int K) {
  return nv ? (size_t)E * amax_parts(E, (int64_t)N * (K / 16)) * sizeof(uint32_t) : 0;
}

hipError_t launch_quant_fp4(const uint16_t* x, bool nv, int E, int N, int K, uint8_t* B, uint8_t* SB, float* gs,
                            uint32_t* work, hipStream_t stream) {
  const int64_t units = (int64_t)N * (K / 16);
  if (!nv) {
    const int64_t all = units * E;
    return in_launches((all + Q_THREADS - 1) / Q_THREADS, Q_THREADS, [&](int64_t b, int64_t n) {
      hipLaunchKernelGGL(quant_mx_kernel, dim3((unsigned)n), dim3(Q_THREADS), 0, stream, x, b * Q_THREADS, all, B, SB);
    });
  }
  const int parts = amax_parts(E, units);
  hipError_t e = in_launches((int64_t)E * parts, Q_THREADS, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(expert_amax_kernel, dim3((unsigned)n), dim3(Q_THREADS), 0, stream, x, units, parts, b, work);
  });
  if (e != hipSuccess) return e;
  const int64_t per = (units + Q_THREADS - 1) / Q_THREADS;
  return in_launches(per * E, Q_THREADS, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(quant_nv_kernel, dim3((unsigned)n), dim3(Q_THREADS), 0, stream, x, units, per, b, parts, work,
                       B, SB, gs);
  });
}

hipError_t launch_dequant_fp4(const uint8_t* B, const uint8_t* SB, bool nv, const float* gs, int E, int N, int K,
                              uint16_t* out, hipStream_t stream) {
  const int64_t units = (int64_t)N * (K / 8), per = (units + Q_THREADS - 1) / Q_THREADS;
  const bool past = units * E * 16 > INFINITY_CACHE;
  const auto kernel = nv ? past ? dequant_kernel<true, true> : dequant_kernel<true, false>
                         : past ? dequant_kernel<false, true> : dequant_kernel<false, false>;
  return in_launches(per * E, Q_THREADS, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(Q_THREADS), 0, stream, B, SB, gs, units, per, b, out);
  });
}

hipError_t launch_quant_gather_fp4(const uint16_t* x, int T, int K, const int32_t* row_of_slot, int top_k, int R,
                                   uint8_t* A, uint8_t* SA, hipStream_t stream) {
  const int threads = std::min(Q_THREADS, (K / 16 + 63) / 64 * 64);
  return in_launches(T, threads, [&](int64_t t, int64_t n) {
    hipLaunchKernelGGL(quant_gather_mx_kernel, dim3((unsigned)n), dim3(threads), 0, stream, x + t * K, K,
                       row_of_slot + t * top_k, top_k, R, A, SA);
  });
}

}  // namespace w4a8
