// Router gate: the top_k experts of every token and their weights, and the
// gradient of the logits, gfx950.
//
// Per token, with logits l[0 .. E-1] (order: larger first, equal values by
// lower index, NaN before everything, -inf never selected):
//   softmax          w_i = c e^(l_i - m) / sum over all e of e^(l_e - m)
//   softmax, renorm  w_i = c e^(l_i - m) / sum over the selected
//   sigmoid          w_i = c s(l_i)
//   sigmoid, renorm  w_i = c s(l_i) / sum over the selected of s
// Backward, with g_i = c dw_i:
//   softmax          dl_e = p_e (sum_i g_i [id_i = e] - sum_i g_i p_i)
//   softmax, renorm  dl_i = u_i (g_i - sum_j g_j u_j), u = w / c
//   sigmoid          dl_i = g_i s_i (1 - s_i)
//   sigmoid, renorm  dl_i = u_i (g_i - sum_j g_j u_j) (1 - s_i)
//
// One wave per row of up to 1024 experts; wider rows take one workgroup, 1024
// experts per wave.  A lane holds V consecutive experts, so a lower lane
// always holds lower indexes and the lowest lane of a ballot breaks ties.
#include "swiglu.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

namespace w4a8 {
namespace {

constexpr int GATE_WAVES = 16;   // most waves of a row
constexpr int ROWS_PER_WG = 4;   // rows of a workgroup when a wave serves a row

// Order-preserving integer of a logit: larger float, larger key; NaN above
// +inf, -0 equal to +0; key 0 marks what is already taken or past the row.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xffffffffu) return __builtin_nanf("");
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d, 64));
  return v;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  if (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return ((const float*)p)[i];
}

// The wave's k largest of 64 V keys: lane j ends with pick j's key in `pk`
// and its position (lane V + i) in `pp`; picks past the last key above -inf
// are (0, -1).  Consumes the keys.
template <int V>
__device__ __forceinline__ void wave_topk(uint32_t (&key)[V], int k, uint32_t& pk, int& pp) {
  const int lane = threadIdx.x & 63;
  pk = 0;
  pp = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) { best = key[i]; bi = i; }
    const uint32_t top = wave_max(best);
    if (top <= KEY_NEG_INF) break;
    const int src = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    const int pos = __shfl(lane * V + bi, src, 64);
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == bi) key[i] = 0;
    }
    if (lane == j) { pk = top; pp = pos; }
  }
}

__device__ __forceinline__ float sigmoid(float v) { return __fdiv_rn(1.0f, 1.0f + exp_f32(-v)); }

// s(v) / s(m) for v <= m: s(v) = e^min(v, 0) / (1 + e^-|v|), so the ratio
// neither overflows nor becomes 0 / 0 however negative both logits are.
__device__ __forceinline__ float sigmoid_ratio(float v, float m) {
  return exp_f32(fminf(v, 0.f) - fminf(m, 0.f)) * __fdiv_rn(1.0f + exp_f32(-fabsf(m)), 1.0f + exp_f32(-fabsf(v)));
}

// Weights of the picks (lane j holds pick j), written with their ids.
// all_sum: sum of e^(l - max) over the whole row (softmax without renorm).
__device__ __forceinline__ void write_picks(uint32_t pk, int id, int k, int score, int renorm, float scale,
                                            float all_sum, int32_t* ids, float* weights) {
  const int lane = threadIdx.x & 63;
  const bool ok = id >= 0;
  const float v = key_value(pk);
  const float m = __shfl(v, 0, 64);
  float w = !ok ? 0.f : score == 0 ? exp_f32(v - m) : renorm ? sigmoid_ratio(v, m) : sigmoid(v);
  if (renorm)
    w = __fdiv_rn(w, wave_sum(w));
  else if (score == 0)
    w = __fdiv_rn(w, all_sum);
  if (lane < k) {
    ids[lane] = id;
    weights[lane] = ok ? w * scale : 0.f;
  }
}

template <int V, bool BF16>
__global__ void __launch_bounds__(64 * ROWS_PER_WG)
gate_wave_kernel(const void* __restrict__ logits, int T, int E, int k, int score, int renorm, float scale,
                 int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * ROWS_PER_WG + (threadIdx.x >> 6);
  if (t >= T) return;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    key[i] = e < E ? order_key(load_logit<BF16>(logits, (size_t)t * E + e)) : 0u;
  }
  float all = 0.f;
  if (score == 0 && !renorm) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    const float m = key_value(wave_max(best));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0u && key[i] != KEY_NEG_INF) all += exp_f32(key_value(key[i]) - m);
    all = wave_sum(all);
  }
  uint32_t pk;
  int pp;
  wave_topk<V>(key, k, pk, pp);
  write_picks(pk, pp, k, score, renorm, scale, all, ids + (size_t)t * k, weights + (size_t)t * k);
}

// Rows of more than 1024 experts: every wave ranks its own 1024, wave 0 then
// ranks the waves' picks (at most 16 x 64; kept in wave order, so equal keys
// still go to the lower index).
template <bool BF16>
__global__ void __launch_bounds__(64 * GATE_WAVES)
gate_wide_kernel(const void* __restrict__ logits, int E, int k, int score, int renorm, float scale,
                 int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr int V = 16;
  __shared__ uint32_t s_key[GATE_WAVES * 64];
  __shared__ int s_pos[GATE_WAVES * 64];
  __shared__ uint32_t s_max[GATE_WAVES];
  __shared__ float s_sum[GATE_WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const size_t t = blockIdx.x;
  const int base = wave * 64 * V;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = base + lane * V + i;
    key[i] = e < E ? order_key(load_logit<BF16>(logits, t * E + e)) : 0u;
  }
  if (score == 0 && !renorm) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, key[i]);
    const uint32_t km = wave_max(best);
    const float m = key_value(km);
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0u && key[i] != KEY_NEG_INF) all += exp_f32(key_value(key[i]) - m);
    all = wave_sum(all);
    if (lane == 0) { s_max[wave] = km; s_sum[wave] = all; }
  }
  uint32_t pk;
  int pp;
  wave_topk<V>(key, k, pk, pp);
  if (lane < k) {
    s_key[wave * k + lane] = pk;
    s_pos[wave * k + lane] = pp < 0 ? -1 : base + pp;
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane * V + i;
    key[i] = c < waves * k ? s_key[c] : 0u;
  }
  wave_topk<V>(key, k, pk, pp);
  float all = 0.f;
  if (score == 0 && !renorm) {
    const uint32_t mine = lane < waves ? s_max[lane] : 0u;
    const float m = key_value(wave_max(mine));
    all = mine > KEY_NEG_INF ? s_sum[lane] * exp_f32(key_value(mine) - m) : 0.f;
    all = wave_sum(all);
  }
  const int id = pp < 0 ? -1 : s_pos[pp];
  write_picks(pk, id, k, score, renorm, scale, all, ids + t * k, weights + t * k);
}

__device__ __forceinline__ float block_sum(float v, float* buf, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += buf[w];
  return s;
}
__device__ __forceinline__ float block_max(float v, float* buf, int waves) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  if (waves == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int w = 0; w < waves; ++w) v = fmaxf(v, buf[w]);
  return v;
}

// One row: `waves` waves starting at the caller's, V experts per lane.
template <int V, bool BF16>
__device__ __forceinline__ void gate_backward_row(const void* logits, size_t t, int E, const int32_t* ids,
                                                  const float* dweights, int k, int score, int renorm, float scale,
                                                  void* dlogits, int first, int waves, float* buf) {
  const int lane = threadIdx.x & 63;
  // lane j of every wave holds slot j
  int id = lane < k ? ids[t * k + lane] : -1;
  if (id >= E) id = -1;
  const bool ok = id >= 0;
  const float v = ok ? load_logit<BF16>(logits, t * E + id) : 0.f;
  const float g = ok ? dweights[t * k + lane] * scale : 0.f;
  float l[V], d[V];
  if (score == 0 && !renorm) {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = first + lane * V + i;
      l[i] = e < E ? load_logit<BF16>(logits, t * E + e) : -__builtin_inff();
      m = fmaxf(m, l[i]);
    }
    m = block_max(m, buf, waves);
    const float mm = m == -__builtin_inff() ? 0.f : m;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = exp_f32(l[i] - mm);
      z += l[i];
    }
    z = block_sum(z, buf, waves);
    const float rz = m == -__builtin_inff() ? 0.f : __fdiv_rn(1.0f, z);
    const float dot = wave_sum(ok ? g * (exp_f32(v - mm) * rz) : 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = -dot;
    for (int j = 0; j < k; ++j) {
      const int idj = __shfl(id, j, 64);
      const float gj = __shfl(g, j, 64);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (first + lane * V + i == idj) d[i] += gj;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] *= l[i] * rz;
  } else {
    // 1 - s from e^v: no cancellation for large logits
    const float c = score == 0 ? 1.f : __fdiv_rn(1.0f, 1.0f + exp_f32(v));
    float dv;
    if (renorm) {
      float m = ok ? v : -__builtin_inff();
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
      const float r = !ok ? 0.f : score == 0 ? exp_f32(v - m) : sigmoid_ratio(v, m);
      const float u = __fdiv_rn(r, wave_sum(r));
      dv = u * (g - wave_sum(ok ? g * u : 0.f)) * c;
    } else {
      dv = g * sigmoid(v) * c;
    }
    if (!ok) dv = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    for (int j = 0; j < k; ++j) {
      const int idj = __shfl(id, j, 64);
      const float dj = __shfl(dv, j, 64);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (first + lane * V + i == idj) d[i] += dj;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = first + lane * V + i;
    if (e >= E) continue;
    if (BF16)
      ((__bf16*)dlogits)[t * E + e] = (__bf16)d[i];
    else
      ((float*)dlogits)[t * E + e] = d[i];
  }
}

template <int V, bool BF16>
__global__ void __launch_bounds__(64 * ROWS_PER_WG)
gate_backward_wave_kernel(const void* __restrict__ logits, int T, int E, const int32_t* __restrict__ ids,
                          const float* __restrict__ dweights, int k, int score, int renorm, float scale,
                          void* __restrict__ dlogits) {
  const int64_t t = (int64_t)blockIdx.x * ROWS_PER_WG + (threadIdx.x >> 6);
  if (t >= T) return;
  gate_backward_row<V, BF16>(logits, (size_t)t, E, ids, dweights, k, score, renorm, scale, dlogits, 0, 1, nullptr);
}

template <bool BF16>
__global__ void __launch_bounds__(64 * GATE_WAVES)
gate_backward_wide_kernel(const void* __restrict__ logits, int E, const int32_t* __restrict__ ids,
                          const float* __restrict__ dweights, int k, int score, int renorm, float scale,
                          void* __restrict__ dlogits) {
  __shared__ float buf[GATE_WAVES];
  gate_backward_row<16, BF16>(logits, blockIdx.x, E, ids, dweights, k, score, renorm, scale, dlogits,
                              (threadIdx.x >> 6) * 1024, blockDim.x >> 6, buf);
}

template <bool BF16>
void launch_fwd(const void* logits, int T, int E, int k, int score, int renorm, float scale, int32_t* ids,
                float* weights, hipStream_t st) {
  const dim3 grid((T + ROWS_PER_WG - 1) / ROWS_PER_WG), block(64 * ROWS_PER_WG);
#define W4A8_GATE(V) \
  hipLaunchKernelGGL((gate_wave_kernel<V, BF16>), grid, block, 0, st, logits, T, E, k, score, renorm, scale, ids, weights)
  if (E <= 64) W4A8_GATE(1);
  else if (E <= 128) W4A8_GATE(2);
  else if (E <= 256) W4A8_GATE(4);
  else if (E <= 512) W4A8_GATE(8);
  else if (E <= 1024) W4A8_GATE(16);
  else
    hipLaunchKernelGGL((gate_wide_kernel<BF16>), dim3(T), dim3(64 * ((E + 1023) / 1024)), 0, st, logits, E, k, score,
                       renorm, scale, ids, weights);
#undef W4A8_GATE
}

template <bool BF16>
void launch_bwd(const void* logits, int T, int E, const int32_t* ids, const float* dweights, int k, int score,
                int renorm, float scale, void* dlogits, hipStream_t st) {
  const dim3 grid((T + ROWS_PER_WG - 1) / ROWS_PER_WG), block(64 * ROWS_PER_WG);
#define W4A8_GATE(V)                                                                                                \
  hipLaunchKernelGGL((gate_backward_wave_kernel<V, BF16>), grid, block, 0, st, logits, T, E, ids, dweights, k, score, \
                     renorm, scale, dlogits)
  if (E <= 64) W4A8_GATE(1);
  else if (E <= 128) W4A8_GATE(2);
  else if (E <= 256) W4A8_GATE(4);
  else if (E <= 512) W4A8_GATE(8);
  else if (E <= 1024) W4A8_GATE(16);
  else
    hipLaunchKernelGGL((gate_backward_wide_kernel<BF16>), dim3(T), dim3(64 * ((E + 1023) / 1024)), 0, st, logits, E,
                       ids, dweights, k, score, renorm, scale, dlogits);
#undef W4A8_GATE
}

}  // namespace

hipError_t launch_topk_gate(const void* logits, bool bf16, int T, int E, int k, int score, int renorm, float scale,
                            int32_t* ids, float* weights, hipStream_t stream) {
  if (bf16)
    launch_fwd<true>(logits, T, E, k, score, renorm, scale, ids, weights, stream);
  else
    launch_fwd<false>(logits, T, E, k, score, renorm, scale, ids, weights, stream);
  return hipGetLastError();
}

hipError_t launch_topk_gate_backward(const void* logits, bool bf16, int T, int E, const int32_t* ids,
                                     const float* dweights, int k, int score, int renorm, float scale, void* dlogits,
                                     hipStream_t stream) {
  if (bf16)
    launch_bwd<true>(logits, T, E, ids, dweights, k, score, renorm, scale, dlogits, stream);
  else
    launch_bwd<false>(logits, T, E, ids, dweights, k, score, renorm, scale, dlogits, stream);
  return hipGetLastError();
}

}  // namespace w4a8
