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
// Rows of up to 64 experts: one expert per lane, one row per wave or two in
// its halves, k rounds of a wave maximum.  Wider rows take one workgroup, 4 to
// 24 experts in a lane's registers (up to 1536 per wave); there the k-th
// largest of 64 group maxima bounds the selection from below, the few experts
// that reach it are collected in LDS and ranked by counting.  (Ranking by k rounds
// of a maximum over all of a lane's experts took 53 us on 2047 x 6144.)
//
// What it measured in the kernel: 64 x 32 3.0 us and the gradient of 16384 x
// 32 4.7 us, both at the length of a launch and one trip to memory; 2047 x
// 6144 bf16 9.4 to 10.8 us (25 MB: 2.5 TB/s; 17 us for the softmax over all),
// bound by the three barriers of a row and the rounds of a maximum between
// them, with 8 rows on a CU.  The gradient of 2047 x 6144 bf16, a call: 12.6
// us for the sigmoid (25 MB written, only the selected logits read), 20.8 us
// for the softmax over all (50 MB: 2.4 TB/s).
#include "swiglu.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <type_traits>

namespace w4a8 {
namespace {

constexpr int GATE_WAVES = 16;   // most waves of a row
constexpr int GATE_CAND = 64;    // experts that are ranked by counting, one per lane
constexpr int ROWS_PER_WG = 4;   // waves of a workgroup of narrow rows

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

// Sum and maximum over the W = 64 lanes of a wave or the 32 of its halves, in
// every lane: DPP row shifts, then row broadcasts (lanes without a source
// read 0).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int W>
__device__ __forceinline__ uint32_t last_lane(uint32_t v) {
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  if (W == 64) return hi;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)v, 31);
  return (threadIdx.x & 32) ? hi : lo;
}
template <int W>
__device__ __forceinline__ float row_sum(float v) {
  v += __uint_as_float(dpp0<0x111, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(dpp0<0x112, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(dpp0<0x114, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(dpp0<0x118, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(dpp0<0x142, 0xa>(__float_as_uint(v)));
  if (W == 64) v += __uint_as_float(dpp0<0x143, 0xc>(__float_as_uint(v)));
  return __uint_as_float(last_lane<W>(__float_as_uint(v)));
}
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp0<0x111, 0xf>(v));
  v = max(v, dpp0<0x112, 0xf>(v));
  v = max(v, dpp0<0x114, 0xf>(v));
  v = max(v, dpp0<0x118, 0xf>(v));
  v = max(v, dpp0<0x142, 0xa>(v));
  if (W == 64) v = max(v, dpp0<0x143, 0xc>(v));
  return last_lane<W>(v);
}
// first lane of the row (0 .. W-1) whose p holds, -1 if none
template <int W>
__device__ __forceinline__ int row_first(bool p) {
  const uint64_t m = __ballot(p);
  if (W == 64) return __ffsll((unsigned long long)m) - 1;
  return __ffs((threadIdx.x & 32) ? (uint32_t)(m >> 32) : (uint32_t)m) - 1;
}
// v of lane i of the row
template <int W>
__device__ __forceinline__ uint32_t row_get(uint32_t v, int i) {
  return (uint32_t)__shfl((int)v, (threadIdx.x & (64 - W)) + i, 64);
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
  if (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return ((const float*)p)[i];
}

__device__ __forceinline__ float sigmoid(float v) { return __fdiv_rn(1.0f, 1.0f + exp_f32(-v)); }

// s(v) / s(m) for v <= m: s(v) = e^min(v, 0) / (1 + e^-|v|), so the ratio
// neither overflows nor becomes 0 / 0 however negative both logits are.
__device__ __forceinline__ float sigmoid_ratio(float v, float m) {
  return exp_f32(fminf(v, 0.f) - fminf(m, 0.f)) * __fdiv_rn(1.0f + exp_f32(-fabsf(m)), 1.0f + exp_f32(-fabsf(v)));
}

// Weights of the picks (lane j of the row holds pick j), written with their
// ids.  all_sum: sum of e^(l - max) over the whole row (softmax without renorm).
template <int W>
__device__ __forceinline__ void write_picks(uint32_t pk, int id, int k, int score, int renorm, float scale,
                                            float all_sum, int32_t* ids, float* weights) {
  const int lane = threadIdx.x & (W - 1);
  const bool ok = id >= 0;
  const float v = key_value(pk);
  const float m = __uint_as_float(row_get<W>(__float_as_uint(v), 0));
  float w = !ok ? 0.f : score == 0 ? exp_f32(v - m) : renorm ? sigmoid_ratio(v, m) : sigmoid(v);
  if (renorm)
    w = __fdiv_rn(w, row_sum<W>(w));
  else if (score == 0)
    w = __fdiv_rn(w, all_sum);
  if (lane < k) {
    ids[lane] = id;
    weights[lane] = ok ? w * scale : 0.f;
  }
}

// Rows of up to W experts, 64 / W of them per wave.
template <int W, bool BF16>
__global__ void __launch_bounds__(64 * ROWS_PER_WG)
gate_narrow_kernel(const void* __restrict__ logits, int T, int E, int k, int score, int renorm, float scale,
                   int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & (W - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / W) + threadIdx.x / W;
  const bool live = row < T;
  const size_t t = live ? row : 0;
  uint32_t key = live && lane < E ? order_key(load_logit<BF16>(logits, t * E + lane)) : 0u;
  float all = 0.f;
  if (score == 0 && !renorm) {
    const float m = key_value(row_max<W>(key));
    all = row_sum<W>(key > KEY_NEG_INF ? exp_f32(key_value(key) - m) : 0.f);
  }
  uint32_t pk = 0;
  int id = -1;
  for (int j = 0; j < k; ++j) {
    const uint32_t top = row_max<W>(key);
    if (!__ballot(top > KEY_NEG_INF)) break;
    const int src = row_first<W>(key == top);   // the lowest of equals
    if (lane == j && top > KEY_NEG_INF) pk = top, id = src;
    if (lane == src) key = 0;
  }
  if (!live) return;
  write_picks<W>(pk, id, k, score, renorm, scale, all, ids + t * k, weights + t * k);
}

// V experts per lane as V / VEC loads of up to 16 bytes: element (c, j) of a
// lane is expert base + (64 c + lane) VEC + j.
template <int V, bool BF16>
struct Lane {
  static constexpr int VEC = BF16 ? (V < 8 ? V : 8) : 4;
  static __device__ __forceinline__ int expert(int base, int i) {
    return base + (64 * (i / VEC) + (int)(threadIdx.x & 63)) * VEC + i % VEC;
  }
  static __device__ __forceinline__ void load(const void* logits, size_t row, int E, int base, float pad, float (&l)[V]) {
#pragma unroll
    for (int c = 0; c < V / VEC; ++c) {
      const int e = expert(base, c * VEC);
      if (e + VEC <= E) {   // rows start at any element: the loads need no alignment
        uint32_t w[BF16 ? VEC / 2 : VEC];
        __builtin_memcpy(w, (const char*)logits + (row + e) * (BF16 ? 2 : 4), sizeof(w));
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          l[c * VEC + j] = __uint_as_float(!BF16 ? w[j] : (j & 1) ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) l[c * VEC + j] = e + j < E ? load_logit<BF16>(logits, row + e + j) : pad;
      }
    }
  }
  static __device__ __forceinline__ void store(void* out, size_t row, int E, int base, const float (&d)[V]) {
#pragma unroll
    for (int c = 0; c < V / VEC; ++c) {
      const int e = expert(base, c * VEC);
      if (BF16) {
        uint16_t w[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = __builtin_bit_cast(uint16_t, (__bf16)d[c * VEC + j]);
        if (e + VEC <= E)
          __builtin_memcpy((uint16_t*)out + row + e, w, sizeof(w));
        else
          for (int j = 0; j < VEC; ++j)
            if (e + j < E) ((uint16_t*)out)[row + e + j] = w[j];
      } else {
        if (e + VEC <= E)
          __builtin_memcpy((float*)out + row + e, &d[c * VEC], 4 * VEC);
        else
          for (int j = 0; j < VEC; ++j)
            if (e + j < E) ((float*)out)[row + e + j] = d[c * VEC + j];
      }
    }
  }
};

// The wave's k largest of its lanes' keys, equal keys by ascending expert:
// lane j ends with pick j (0, -1 past the last key above -inf).
template <int V, bool BF16>
__device__ __forceinline__ void wave_topk(uint32_t (&key)[V], int base, int k, uint32_t& pk, int& id) {
  const int lane = threadIdx.x & 63;
  pk = 0;
  id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) { best = key[i]; bi = i; }
    const uint32_t top = row_max<64>(best);
    if (top <= KEY_NEG_INF) break;
    int e = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i == bi) e = Lane<V, BF16>::expert(base, i);
    const int first = ~(int)row_max<64>(best == top ? ~(uint32_t)e : 0u);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (best == top && e == first && i == bi) key[i] = 0;
    if (lane == j) pk = top, id = first;
  }
}

template <int V, bool BF16>
__global__ void __launch_bounds__(64 * GATE_WAVES, 8)
gate_kernel(const void* __restrict__ logits, int E, int k, int score, int renorm, float scale,
            int32_t* __restrict__ ids, float* __restrict__ weights) {
  __shared__ uint32_t s_max[GATE_WAVES * 64];   // the lanes' maxima; the waves' picks
  __shared__ int s_id[GATE_WAVES * 64];
  __shared__ float s_sum[GATE_WAVES];
  __shared__ uint32_t s_bound, s_top;
  __shared__ int s_count;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const size_t t = blockIdx.x;
  const int base = wave * 64 * V;
  uint32_t key[V], best = 0;
  {
    float l[V];
    Lane<V, BF16>::load(logits, t * E, E, base, -__builtin_inff(), l);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      key[i] = order_key(l[i]);
      best = max(best, key[i]);
    }
  }
  s_max[threadIdx.x] = best;
  if (threadIdx.x == 0) s_count = 0;
  __syncthreads();
  if (wave == 0) {   // the k-th largest of 64 group maxima (a group: one lane of every wave)
    uint32_t group = best, bound = 0, top0 = 0;
    for (int w = 1; w < waves; ++w) group = max(group, s_max[w * 64 + lane]);
    for (int j = 0; j < k; ++j) {
      const uint32_t top = row_max<64>(group);
      if (j == 0) top0 = top;
      bound = max(top, KEY_NEG_INF + 1);
      if (top <= KEY_NEG_INF) break;
      if (lane == row_first<64>(group == top)) group = 0;
    }
    if (lane == 0) s_bound = bound, s_top = top0;
  }
  __syncthreads();
  const uint32_t bound = s_bound;
  if (best >= bound) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] >= bound) {
        const int at = atomicAdd(&s_count, 1);   // any order: they are ranked by key and expert
        if (at < GATE_CAND) s_max[at] = key[i], s_id[at] = Lane<V, BF16>::expert(base, i);
      }
  }
  if (score == 0 && !renorm) {
    const float m = key_value(s_top);
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) all += key[i] > KEY_NEG_INF ? exp_f32(key_value(key[i]) - m) : 0.f;
    all = row_sum<64>(all);
    if (lane == 0) s_sum[wave] = all;
  }
  __syncthreads();
  const int n = s_count;
  uint32_t pk = 0;
  int id = -1;
  if (n <= GATE_CAND) {
    if (wave != 0) return;
    const uint32_t mine = lane < n ? s_max[lane] : 0u;
    const int e = lane < n ? s_id[lane] : -1;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, j);
      const int oe = __builtin_amdgcn_readlane(e, j);
      rank += other > mine || (other == mine && oe < e) ? 1 : 0;
    }
    // pick j to lane j
    if (lane < n && rank < k) s_max[64 + rank] = mine, s_id[64 + rank] = e;
    __builtin_amdgcn_wave_barrier();
    if (lane < min(n, k)) pk = s_max[64 + lane], id = s_id[64 + lane];
  } else {
    // many picks, or many equal keys: every wave ranks its own, wave 0 the
    // waves' picks (at most 16 x 64, a lane's 16 in wave order)
    wave_topk<V, BF16>(key, base, k, pk, id);
    __syncthreads();
    if (lane < k) s_max[wave * k + lane] = pk, s_id[wave * k + lane] = id;
    __syncthreads();
    if (wave != 0) return;
    if (waves > 1) {
      constexpr int M = GATE_WAVES;
      uint32_t mk[M];
      const int total = waves * k;
#pragma unroll
      for (int i = 0; i < M; ++i) mk[i] = lane * M + i < total ? s_max[lane * M + i] : 0u;
      // equal keys: a lower place holds a lower expert
      pk = 0;
      id = -1;
      for (int j = 0; j < k; ++j) {
        uint32_t b = mk[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < M; ++i)
          if (mk[i] > b) { b = mk[i]; bi = i; }
        const uint32_t top = row_max<64>(b);
        if (top <= KEY_NEG_INF) break;
        const int src = row_first<64>(b == top);
        const int place = (int)row_get<64>((uint32_t)(lane * M + bi), src);
        if (lane == src) {
#pragma unroll
          for (int i = 0; i < M; ++i)
            if (i == bi) mk[i] = 0;
        }
        if (lane == j) pk = top, id = s_id[place];
      }
    }
  }
  float all = 0.f;
  if (score == 0 && !renorm) all = row_sum<64>(lane < waves ? s_sum[lane] : 0.f);
  write_picks<64>(pk, id, k, score, renorm, scale, all, ids + t * k, weights + t * k);
}

// What a slot's lane adds at its expert (lane j of the row holds slot j, v its
// logit, g = scale * dweight): dv, for every score but the softmax over all.
template <int W>
__device__ __forceinline__ float slot_gradient(bool ok, float v, float g, int score, int renorm) {
  // 1 - s from e^v: no cancellation for large logits
  const float c = score == 0 ? 1.f : __fdiv_rn(1.0f, 1.0f + exp_f32(v));
  float dv;
  if (renorm) {
    const float m = key_value(row_max<W>(ok ? order_key(v) : 0u));
    const float r = !ok ? 0.f : score == 0 ? exp_f32(v - m) : sigmoid_ratio(v, m);
    const float u = __fdiv_rn(r, row_sum<W>(r));
    dv = u * (g - row_sum<W>(ok ? g * u : 0.f)) * c;
  } else {
    dv = g * sigmoid(v) * c;
  }
  return ok ? dv : 0.f;
}

// Rows of up to W experts, 64 / W of them per wave (k <= W).
template <int W, bool BF16>
__global__ void __launch_bounds__(64 * ROWS_PER_WG)
gate_backward_narrow_kernel(const void* __restrict__ logits, int T, int E, const int32_t* __restrict__ ids,
                            const float* __restrict__ dweights, int k, int score, int renorm, float scale,
                            void* __restrict__ dlogits) {
  const int lane = threadIdx.x & (W - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / W) + threadIdx.x / W;
  const bool live = row < T;
  const size_t t = live ? row : 0;
  int id = live && lane < k ? ids[t * k + lane] : -1;
  float g = live && lane < k ? dweights[t * k + lane] : 0.f;
  const float l = live && lane < E ? load_logit<BF16>(logits, t * E + lane) : -__builtin_inff();
  if (id >= E) id = -1;
  const bool ok = id >= 0;
  g = ok ? g * scale : 0.f;
  const float v = __uint_as_float(row_get<W>(__float_as_uint(l), ok ? id : 0));
  float d = 0.f, add = g, p = 1.f;
  if (score == 0 && !renorm) {
    const float m = key_value(row_max<W>(order_key(l)));
    const float mm = m == -__builtin_inff() ? 0.f : m;
    const float x = exp_f32(l - mm);
    const float z = row_sum<W>(x);
    p = m == -__builtin_inff() ? 0.f : x * __fdiv_rn(1.0f, z);
    const float pv = __uint_as_float(row_get<W>(__float_as_uint(p), ok ? id : 0));
    d = -row_sum<W>(ok ? g * pv : 0.f);
  } else {
    add = slot_gradient<W>(ok, v, g, score, renorm);
  }
  for (int j = 0; j < k; ++j) {
    const int idj = (int)row_get<W>((uint32_t)id, j);
    const float a = __uint_as_float(row_get<W>(__float_as_uint(add), j));
    if (lane == idj) d += a;
  }
  d *= p;
  if (!live || lane >= E) return;
  if (BF16)
    ((__bf16*)dlogits)[t * E + lane] = (__bf16)d;
  else
    ((float*)dlogits)[t * E + lane] = d;
}

__device__ __forceinline__ float block_sum(float v, float* buf, int waves) {
  v = row_sum<64>(v);
  if (waves == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < waves; ++w) s += buf[w];
  return s;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, float* buf, int waves) {
  v = row_max<64>(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  for (int w = 0; w < waves; ++w) v = max(v, __float_as_uint(buf[w]));
  return v;
}

// One row per workgroup.
template <int V, bool BF16>
__global__ void __launch_bounds__(64 * GATE_WAVES)
gate_backward_kernel(const void* __restrict__ logits, int E, const int32_t* __restrict__ ids,
                     const float* __restrict__ dweights, int k, int score, int renorm, float scale,
                     void* __restrict__ dlogits) {
  __shared__ float buf[GATE_WAVES];
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const size_t t = blockIdx.x;
  const int base = (threadIdx.x >> 6) * 64 * V;
  // lane j of every wave holds slot j
  int id = lane < k ? ids[t * k + lane] : -1;
  float l[V], d[V];
  if (score == 0 && !renorm) Lane<V, BF16>::load(logits, t * E, E, base, -__builtin_inff(), l);
  if (id >= E) id = -1;
  const bool ok = id >= 0;
  const float v = ok ? load_logit<BF16>(logits, t * E + id) : 0.f;
  const float g = ok ? dweights[t * k + lane] * scale : 0.f;
  float add = g;
  if (score == 0 && !renorm) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) best = max(best, order_key(l[i]));
    const float m = key_value(block_max(best, buf, waves));
    const bool none = m == -__builtin_inff();
    const float mm = none ? 0.f : m;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = exp_f32(l[i] - mm);
      z += l[i];
    }
    z = block_sum(z, buf, waves);
    const float rz = none ? 0.f : __fdiv_rn(1.0f, z);
    const float dot = row_sum<64>(ok ? g * (exp_f32(v - mm) * rz) : 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] *= rz;
      d[i] = -dot;
    }
  } else {
    add = slot_gradient<64>(ok, v, g, score, renorm);
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = 1.f, d[i] = 0.f;
  }
  for (int j = 0; j < k; ++j) {
    const int idj = __builtin_amdgcn_readlane(id, j) - base;
    const float a = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(add), j));
    if ((unsigned)idj < 64u * V) {   // in this wave
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (Lane<V, BF16>::expert(0, i) == idj) d[i] += a;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] *= l[i];
  Lane<V, BF16>::store(dlogits, t * E, E, base, d);
}

// Lanes and experts per lane for E experts.  Past 1024: 24 per lane in 64
// registers, so that 8 rows of 6144 fit on a CU at once (2047 x 6144 bf16: 10.3
// us; 12.3 with 16 per lane, 13.0 with 32).
#define W4A8_GATE_ROWS(NARROW, ROW)                                                                           \
  if (E <= 32 && k <= 32) {                                                                                   \
    NARROW(32)                                                                                                \
  } else if (E <= 64) {                                                                                       \
    NARROW(64)                                                                                                \
  } else if (E <= 256) {                                                                                      \
    ROW(4)                                                                                                    \
  } else if (E <= 512) {                                                                                      \
    ROW(8)                                                                                                    \
  } else if (E <= 1024) {                                                                                     \
    ROW(16)                                                                                                   \
  } else {                                                                                                    \
    ROW(24)                                                                                                   \
  }

unsigned narrow_grid(int64_t T, int W) { return (unsigned)((T * W + 64 * ROWS_PER_WG - 1) / (64 * ROWS_PER_WG)); }
unsigned row_threads(int E, int V) { return 64u * ((E + 64 * V - 1) / (64 * V)); }
template <bool BF16, typename P>
P* row_of(P* logits, int64_t t, int E) {
  typedef typename std::conditional<std::is_const<P>::value, const char, char>::type Byte;
  return (Byte*)logits + (size_t)t * E * (BF16 ? 2 : 4);
}

template <bool BF16>
hipError_t launch_fwd(const void* logits, int T, int E, int k, int score, int renorm, float scale, int32_t* ids,
                      float* weights, hipStream_t st) {
#define NARROW(W)                                                                                                \
  return in_launches(T, W, [&](int64_t t, int64_t n) {                                                           \
    hipLaunchKernelGGL((gate_narrow_kernel<W, BF16>), dim3(narrow_grid(n, W)), dim3(64 * ROWS_PER_WG), 0, st,    \
                       row_of<BF16>(logits, t, E), (int)n, E, k, score, renorm, scale, ids + t * k, weights + t * k); \
  });
#define ROW(V)                                                                                                   \
  return in_launches(T, row_threads(E, V), [&](int64_t t, int64_t n) {                                           \
    hipLaunchKernelGGL((gate_kernel<V, BF16>), dim3((unsigned)n), dim3(row_threads(E, V)), 0, st,                \
                       row_of<BF16>(logits, t, E), E, k, score, renorm, scale, ids + t * k, weights + t * k);    \
  });
  W4A8_GATE_ROWS(NARROW, ROW)
#undef NARROW
#undef ROW
}

template <bool BF16>
hipError_t launch_bwd(const void* logits, int T, int E, const int32_t* ids, const float* dweights, int k, int score,
                      int renorm, float scale, void* dlogits, hipStream_t st) {
#define NARROW(W)                                                                                                \
  return in_launches(T, W, [&](int64_t t, int64_t n) {                                                           \
    hipLaunchKernelGGL((gate_backward_narrow_kernel<W, BF16>), dim3(narrow_grid(n, W)), dim3(64 * ROWS_PER_WG), 0, st, \
                       row_of<BF16>(logits, t, E), (int)n, E, ids + t * k, dweights + t * k, k, score, renorm, scale, \
                       row_of<BF16>(dlogits, t, E));                                                             \
  });
#define ROW(V)                                                                                                   \
  return in_launches(T, row_threads(E, V), [&](int64_t t, int64_t n) {                                           \
    hipLaunchKernelGGL((gate_backward_kernel<V, BF16>), dim3((unsigned)n), dim3(row_threads(E, V)), 0, st,       \
                       row_of<BF16>(logits, t, E), E, ids + t * k, dweights + t * k, k, score, renorm, scale,    \
                       row_of<BF16>(dlogits, t, E));                                                             \
  });
  W4A8_GATE_ROWS(NARROW, ROW)
#undef NARROW
#undef ROW
}
#undef W4A8_GATE_ROWS

}  // namespace

hipError_t launch_topk_gate(const void* logits, bool bf16, int T, int E, int k, int score, int renorm, float scale,
                            int32_t* ids, float* weights, hipStream_t stream) {
  if (bf16) return launch_fwd<true>(logits, T, E, k, score, renorm, scale, ids, weights, stream);
  return launch_fwd<false>(logits, T, E, k, score, renorm, scale, ids, weights, stream);
}

hipError_t launch_topk_gate_backward(const void* logits, bool bf16, int T, int E, const int32_t* ids,
                                     const float* dweights, int k, int score, int renorm, float scale, void* dlogits,
                                     hipStream_t stream) {
  if (bf16) return launch_bwd<true>(logits, T, E, ids, dweights, k, score, renorm, scale, dlogits, stream);
  return launch_bwd<false>(logits, T, E, ids, dweights, k, score, renorm, scale, dlogits, stream);
}

}  // namespace w4a8
