// Products of single tokens with 4-bit weights and group scales, gfx950:
//
//   y[s, n] = bf16( gs[e] * sum_k x[row(s), k] * (q(e, n, k) - z(e, n, k / g)) * s(e, n, k / g) )
//
// e = the slot's expert (0 without ids), row(s) = s / (S / X).  MXFP4: q an
// E2M1 value, s = 2^(code - 127) per 32 K; NVFP4: s an E4M3 value per 16 K;
// INT4: q a code 0 .. 15, z its zero point (8 when none are given), s bf16
// per 32, 64 or 128 K.  No zero point for the first two.
//
// Bound by the weights' bytes: an expert that some slot names is read once per
// item, up to 16 of its slots (launch_waves: at most twice the mean number of
// slots per expert, at least four), so slots that crowd on few experts read
// these more than once.  matvec_kernel (below) is the path;
// matvec_plain_kernel serves rows shorter than one of its steps, rows that do
// not fit in LDS and experts of 4 GB and more.
#include "w4a8_device.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

namespace w4a8 {
namespace {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float e2m1(uint32_t c) {
  const float mag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  const float v = mag[c & 7];
  return (c & 8) ? -v : v;
}

// E8M0 code -> 2^(c - 127) (code 0: the subnormal 2^-127; 0xFF: NaN).
__device__ __forceinline__ float e8m0(uint32_t c) {
  uint32_t b = c << 23;
  b = c == 0 ? 0x00400000u : b;
  b = c == 0xff ? 0x7fc00000u : b;
  return __uint_as_float(b);
}

enum { F_MX = 0, F_NV = 1, F_INT = 2 };

template <int FMT>
__device__ __forceinline__ float group_scale(const void* p, size_t i) {
  if (FMT == F_MX) return e8m0(((const uint8_t*)p)[i]);
  if (FMT == F_NV) return __builtin_amdgcn_cvt_pk_f32_fp8((int)((const uint8_t*)p)[i], false)[0];
  return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}

// One output by the definition in 64 bits, in every lane of the wave: for
// sums that fp32 does not hold on the way (MXFP4 scales of 2^126 and 2^127,
// whose weights are past bf16 and fp32; sums of x q before a small scale;
// INT4's 16 + q) or in which an infinity met a weight's offset.  col = e N + n.
template <int FMT>
__device__ __forceinline__ float exact_output(const MatvecArgs& a, size_t col, const uint16_t* xr, float gs) {
  const int lane = threadIdx.x & 63;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(a.B + col * (size_t)(a.K >> 1));
  double acc = 0.0;
  for (int c = lane; c < a.K / 8; c += 64) {
    const size_t gi = col * (size_t)(a.K / a.group) + (8 * c) / a.group;
    double sc;
    if (FMT == F_MX) {
      const uint32_t code = ((const uint8_t*)a.SB)[gi];
      sc = code == 0xff ? __builtin_nan("") : __builtin_bit_cast(double, (uint64_t)(code + 896) << 52);
    } else {
      sc = group_scale<FMT>(a.SB, gi);
    }
    const float z = FMT != F_INT ? 0.f : a.zeros ? (float)a.zeros[gi] : 8.f;
    const uint32_t v = w[c];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t q = (v >> (4 * i)) & 15u;
      const double x = __uint_as_float((uint32_t)xr[8 * c + i] << 16);
      acc += x * ((FMT == F_INT ? (float)q - z : e2m1(q)) * sc);
    }
  }
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) acc += __shfl_xor(acc, i, 64);
  return (float)(acc * gs);
}

// exponent all ones: infinite or NaN
__device__ __forceinline__ bool not_finite(uint16_t bf16) { return (bf16 & 0x7f80u) == 0x7f80u; }

// One wave per (slot, column).
template <int FMT>
__global__ void __launch_bounds__(256)
matvec_plain_kernel(const MatvecArgs a) {
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int s = blockIdx.y;
  if (n >= a.N) return;
  const int e = a.ids ? a.ids[s] : 0;
  uint16_t out = 0;
  if (e >= 0 && e < a.E) {
    float acc = 0.f;
    const size_t col = (size_t)e * a.N + n;
    const uint16_t* xr = a.x + (size_t)((s * a.per_row_inv) >> 16) * a.K;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a.B + col * (size_t)(a.K >> 1));
    for (int c = lane; c < a.K / 8; c += 64) {  // 8 weights: inside one group
      const size_t gi = col * (size_t)(a.K / a.group) + (8 * c) / a.group;
      const float sc = group_scale<FMT>(a.SB, gi);
      const float z = FMT != F_INT ? 0.f : a.zeros ? (float)a.zeros[gi] : 8.f;
      const uint32_t v = w[c];
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t q = (v >> (4 * i)) & 15u;
        part = fmaf(__uint_as_float((uint32_t)xr[8 * c + i] << 16), FMT == F_INT ? (float)q - z : e2m1(q), part);
      }
      acc = fmaf(part, sc, acc);
    }
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) acc += __shfl_xor(acc, i, 64);
    const float gs = a.gs ? a.gs[e] : 1.0f;
    out = __builtin_bit_cast(uint16_t, (__bf16)(acc * gs));
    if (not_finite(out)) out = __builtin_bit_cast(uint16_t, (__bf16)exact_output<FMT>(a, col, xr, gs));
  }
  if (lane == 0) a.y[(size_t)s * a.N + n] = out;
}

// ---------------------------------------------------------------------------
// The path.  A workgroup takes one item (up to rows_max slots of one expert)
// and a run of its units (16 columns); its four or eight waves share a unit's
// K in steps of 256 (wave w takes steps w, w + waves, ...) and join their
// sums in LDS.
//
// What it measured (calls in a row, weights not in the caches): 8 experts
// 4096 x 6144, one token, MXFP4 18.7 us (107 MB: 5.7 TB/s; alone in a trace
// 20.5), NVFP4 20.0, INT4 per 128 21.0; 64 slots of 32 such experts 64 us (386
// MB: 6.0 TB/s), all 64 on one expert 30 us (13 MB, read by sixteen items,
// mostly from the caches), INT4 37; 65536 x 6144 dense 34.2 us (214 MB: 6.3
// TB/s); 6144 x 6144 dense, 17, 32 and 64 rows: MXFP4 11, 16 and 24 us, INT4
// 21, 32 and 53.  Bound by HBM, after 3 to 4 us of start (ids, x and
// the first weights, each a trip to memory, and code read for the first time
// in the launch).  Four steps in registers instead of three: 2% more on the
// long shapes, 10% less on one row of 6144 x 6144 (more code); four
// workgroups per CU instead of three: 29.2 against 26.8 us on 131072 x 2048.
// Letting the loads past a workgroup's last unit read that unit again: 26.5
// against 25.2 us on 24 NVFP4 slots of 6144 x 2048 (154 against 143 MB read).
//
// Weights: per step a wave reads 16 columns x 128 bytes as two loads of eight
// whole 128-byte lines (lane l: column l / 8, 16-byte piece l % 8, one piece
// = 32 K), DEPTH - 1 steps ahead in registers, and turns them into the matrix
// instruction's operand order through a private 2 KB of LDS: piece p of
// column c at position p ^ (c / 2 % 8), so that neither side has bank
// conflicts.  Lane 16 q + n then holds pieces 2q and 2q + 1 of column n, and
// v_mfma_f32_16x16x32_bf16 number j of a piece takes its weights 8j .. 8j + 7.
//
// Weights enter the product exactly: MXFP4 as bf16 with its scale (gfx950's
// scaled conversion), NVFP4 as bf16 E2M1 values, INT4 as 16 + q (q in the
// mantissa of 16.0).  For the last two the scales differ within the 128 K
// that one instruction sums over (lane groups q hold different pieces), so x
// is laid out block-diagonally: operand row 4t + p holds token t in lane
// group q = p and zeros in the others; the result then has one sum per
// (token, lane group), and the scales (and the zero points, as (16 + z) times
// the sum of x over the piece) are applied to it in fp32.  Four tokens per
// instruction; MXFP4 takes sixteen.
//
// What fp32 or bf16 do not hold on that way shows as an output that is not
// finite (infinity and NaN never leave a sum again): MXFP4 weights of 2^128
// and more, sums of x q ahead of a small scale, an infinity in x times 16 + q
// less the same times 16 + z.  A wave notes such outputs and computes them
// once more at the end, by exact_output.
//
// x (the rows of the unit's expert) is in LDS as bf16, zeros past K.  Where K
// is no multiple of 256 the last step starts at K - 256: what it repeats
// meets zeros in x.
// ---------------------------------------------------------------------------
constexpr int MV_STEP = 256;              // K per step of a wave
constexpr int MV_WBUF = 2048;             // a wave's LDS for one step of weights
constexpr int MV_X_PAD = 16;              // rows of x start 16 bytes apart modulo 256

// bytes of LDS: weights, partial sums (two units), zeros, slots, x, sums of x
__host__ __device__ inline int mv_row_bytes(int steps) { return steps * (MV_STEP * 2) + MV_X_PAD; }
__host__ __device__ inline int mv_lds_bytes(int waves, int steps, int rows) {
  return waves * MV_WBUF + 2 * waves * rows * 16 * 4 + 128 + 64 * 4 + rows * (mv_row_bytes(steps) + steps * 32);
}

// Workgroups that the registers leave room for on a CU, and the steps of
// weights that a wave holds in registers.
__host__ __device__ constexpr int mv_per_cu(int waves, int tb) { return waves == 8 ? 1 : tb == 4 ? 2 : 3; }
__host__ __device__ constexpr int mv_depth(int waves) { return waves == 8 ? 4 : 3; }

// Scale data of one step: MXFP4 the codes of the lane's two pieces, NVFP4 the
// column's sixteen codes, INT4 its 256 / GROUP bf16 scales and zero points
// (packed in dwords, as loaded).
template <int FMT, int GROUP>
struct Scales {
  static constexpr int NG = MV_STEP / GROUP;
  static constexpr int BYTES = FMT == F_MX ? 2 : FMT == F_NV ? 16 : 2 * NG;
  uint32_t c[(BYTES + 3) / 4];
  uint32_t z[FMT == F_INT ? (NG + 3) / 4 : 1];
};

__device__ __forceinline__ int wkey(int c) { return (c >> 1) & 7; }

// 8 INT4 codes -> 16 + q as bf16, in the order 0 4 1 5 2 6 3 7
// (nib = 0x00780078 in a scalar register, one16 = 0x41804180 in a vector
// register: two instructions per pair)
__device__ __forceinline__ v4u int4_to_bf16(uint32_t w, uint32_t nib, uint32_t one16) {
  v4u o;
  o[0] = ((w << 3) & nib) | one16;
  o[1] = ((w >> 1) & nib) | one16;
  o[2] = ((w >> 5) & nib) | one16;
  o[3] = ((w >> 9) & nib) | one16;
  return o;
}
__device__ __forceinline__ v4u fp4_to_bf16(uint32_t w, float s) {
  v4u o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return o;
}
__device__ __forceinline__ v4f mfma(v4u x, v4u w, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, w), c, 0, 0, 0);
}

// LDS only: every wave's LDS work done, global loads left in flight
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// 16 bytes per lane from src to LDS at to + 16 * lane (`to` wave-uniform).
// Asm, because for a direct-to-LDS load that the compiler knows of it drains
// every load in flight before the next LDS access; wait_loads waits for it.
__device__ __forceinline__ void load_to_lds(const void* src, uint8_t* to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
               "s"(__builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to))
               : "memory", "m0");
}

// at most N of this wave's loads in flight (they complete in issue order)
template <int N>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// TB: sets of four tokens (MXFP4: one set of sixteen, TB = 1).
template <int FMT, int GROUP, int TB, int MV_WAVES>
__global__ void __launch_bounds__(64 * MV_WAVES, mv_per_cu(MV_WAVES, TB) * MV_WAVES / 4)
matvec_kernel(const MatvecArgs a, int rows_max) {
  constexpr int MV_THREADS = 64 * MV_WAVES, MV_DEPTH = mv_depth(MV_WAVES);
  constexpr bool DIAG = FMT != F_MX;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NP = a.K >> 5;                            // pieces of 32 K
  const int steps = (a.K + MV_STEP - 1) / MV_STEP;
  const int mine = (steps - wave + MV_WAVES - 1) / MV_WAVES;   // this wave's steps of a unit
  const int pitch = mv_row_bytes(steps);
  uint8_t* wbuf = lds + wave * MV_WBUF;
  float* red = reinterpret_cast<float*>(lds + MV_WAVES * MV_WBUF);
  uint8_t* zero = reinterpret_cast<uint8_t*>(red + 2 * MV_WAVES * rows_max * 16);
  int* slots = reinterpret_cast<int*>(zero + 128);
  uint8_t* xs = reinterpret_cast<uint8_t*>(slots + 64);
  float* xsum = reinterpret_cast<float*>(xs + rows_max * pitch);   // [row][steps * 8]
  if (tid < 32) reinterpret_cast<uint32_t*>(zero)[tid] = 0u;

  // the experts that some slot names, in the order of their first slots:
  // `same` = the slots with this lane's expert, by one ballot per bit of the id
  int id = 0;
  if (a.ids) {
    id = lane < a.S ? a.ids[lane] : -1;
    if (id >= a.E) id = -1;
  } else if (lane >= a.S) {
    id = -1;
  }
  uint64_t same = __ballot(id >= 0);
  for (int bit = 1; bit < a.E; bit <<= 1) {
    const uint64_t set = __ballot(id & bit);
    same &= (id & bit) ? set : ~set;
  }
  // an item: up to rows_max slots of one expert; a leader lane (an expert's
  // first slot) holds its expert's items before[..] .. upto[..]
  const bool first = id >= 0 && (same & ((1ull << lane) - 1)) == 0;
  const int mine_items = first ? (__popcll(same) + rows_max - 1) / rows_max : 0;
  const int upto = wave_inclusive_sum(mine_items), before = upto - mine_items;
  const int D = __builtin_amdgcn_readlane(upto, 63);
  const int UB = (a.N + 15) >> 4;                     // units of an expert

  // slots without an expert: zeros
  for (uint64_t m = __ballot(lane < a.S && id < 0); m; m &= m - 1) {
    const int s = __ffsll((unsigned long long)m) - 1;
    for (int64_t n = (int64_t)blockIdx.x * MV_THREADS + tid; n < a.N; n += (int64_t)gridDim.x * MV_THREADS)
      a.y[(size_t)s * a.N + n] = 0;
  }

  uint32_t nib = 0x00780078u, one16 = 0x41804180u;
  asm volatile("" : "+s"(nib), "+v"(one16));
  int parity = 0;
  // every item has an equal number of workgroups, a workgroup one item and a
  // run of its units
  const uint32_t each = D ? gridDim.x / (uint32_t)D : 1u;
  const uint32_t d = blockIdx.x / each, w0 = blockIdx.x - d * each;
  if (d < (uint32_t)D) {
    const uint32_t share = UB / each, more = UB % each;
    const int cb0 = share * w0 + min(w0, more);
    const int nu = share + (w0 < more ? 1u : 0u);
    const int leader = __ffsll((unsigned long long)__ballot(before <= (int)d && (int)d < upto)) - 1;
    const int e = __builtin_amdgcn_readlane(id, leader);
    const uint64_t members = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)same, leader) |
                             (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(same >> 32), leader) << 32;
    const int r0 = ((int)d - __builtin_amdgcn_readlane(before, leader)) * rows_max;
    const int rows = min(rows_max, (int)__popcll(members) - r0);
    const float gs = a.gs ? a.gs[e] : 1.0f;
    const uint8_t* Be = a.B + (uint64_t)(uint32_t)e * a.wexp;
    const uint8_t* Se = (const uint8_t*)a.SB + (uint64_t)(uint32_t)e * a.sexp;
    const uint8_t* Ze = FMT == F_INT && a.zeros ? a.zeros + (uint64_t)(uint32_t)e * a.zexp : nullptr;

    if (nu > 0) {
      {  // every wave writes the same list
        const int rank = __popcll(members & ((1ull << lane) - 1)) - r0;
        if (((members >> lane) & 1) && rank >= 0 && rank < rows) slots[rank] = lane;
      }
      // x into LDS without a register between: 16 bytes per lane, 64 units in a
      // row per instruction; what the last step repeats is zeroed
      const int per_x = steps * 32, turns = (per_x + MV_THREADS - 1) / MV_THREADS;
      uint64_t left = members;
      for (int i = 0; i < r0; ++i) left &= left - 1;
      for (int r = 0; r < rows; ++r, left &= left - 1) {
        const int slot = __ffsll((unsigned long long)left) - 1;
        const uint16_t* xr = a.x + (size_t)((slot * a.per_row_inv) >> 16) * a.K;
        for (int t = 0; t < turns; ++t) {
          const int v = tid + t * MV_THREADS, st = v >> 5;
          const int p = min(8 * st, NP - 8) + ((v >> 2) & 7);
          uint8_t* to = xs + r * pitch + (t * MV_THREADS + wave * 64) * 16;
          if (v < per_x) {
            if (p >= 8 * st)
              load_to_lds(xr + p * 32 + (v & 3) * 8, to);
            else
              *reinterpret_cast<v4u*>(to + lane * 16) = v4u{0u, 0u, 0u, 0u};
          }
        }
      }
      // INT4: each unit's elements in the order 0 4 1 5 2 6 3 7, as
      // int4_to_bf16 has the weights, and the sum of every piece (four lanes)
      // (XR rows at a time)
      auto x_finish = [&]() __attribute__((always_inline)) {
        constexpr int XR = 4;
        for (int r0 = 0; r0 < rows; r0 += XR) {
          for (int v = tid; v < per_x; v += MV_THREADS) {
            v4u w[XR];
            float t[XR];
#pragma unroll
            for (int r = 0; r < XR; ++r)
              w[r] = *reinterpret_cast<const v4u*>(xs + min(r0 + r, rows - 1) * pitch + v * 16);
#pragma unroll
            for (int r = 0; r < XR; ++r) {
              t[r] = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                t[r] += __uint_as_float(w[r][i] << 16) + __uint_as_float(w[r][i] & 0xffff0000u);
              t[r] += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(t[r]), 0xB1, 0xf, 0xf, false));  // lane ^ 1
              t[r] += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(t[r]), 0x4E, 0xf, 0xf, false));  // lane ^ 2
            }
#pragma unroll
            for (int r = 0; r < XR; ++r) {
              if (r0 + r >= rows) break;
              if ((v & 3) == 0) xsum[(r0 + r) * steps * 8 + (v >> 2)] = t[r];
              *reinterpret_cast<v4u*>(xs + (r0 + r) * pitch + v * 16) =
                  v4u{__builtin_amdgcn_perm(w[r][2], w[r][0], 0x05040100u), __builtin_amdgcn_perm(w[r][2], w[r][0], 0x07060302u),
                      __builtin_amdgcn_perm(w[r][3], w[r][1], 0x05040100u), __builtin_amdgcn_perm(w[r][3], w[r][1], 0x07060302u)};
            }
          }
        }
      };

      // loads: a wave-uniform base (unit, step) plus the lane's offset
      v4u wa[MV_DEPTH], wb[MV_DEPTH];
      Scales<FMT, GROUP> sc[MV_DEPTH];
      const uint8_t *ub = nullptr, *us = nullptr, *uz = nullptr;
      uint32_t va = 0, vb = 0, vs = 0, vz = 0;
      auto point = [&](int cb) __attribute__((always_inline)) {
        const int last = a.N - 1 - cb * 16;   // columns past it repeat it
        ub = Be + (uint32_t)cb * 16u * a.wcol;
        us = Se + (uint32_t)cb * 16u * a.scol;
        va = (uint32_t)min(lane >> 3, last) * a.wcol + (lane & 7) * 16;
        vb = (uint32_t)min((lane >> 3) + 8, last) * a.wcol + (lane & 7) * 16;
        vs = (uint32_t)min(lane & 15, last) * a.scol + (FMT == F_MX ? 2 * (lane >> 4) : 0);
        if (FMT == F_INT) {   // without zero points the loads read scales, unused
          uz = Ze ? Ze + (uint32_t)cb * 16u * a.zcol : us;
          vz = (uint32_t)min(lane & 15, last) * a.zcol;
        }
      };
      // loads past the last unit, or of a wave without steps, are never used:
      // every lane reads one place
      auto aside = [&]() __attribute__((always_inline)) {
        va = 0;
        vb = 0;
        vs = 0;
        if (FMT == F_INT) vz = 0;
      };
      auto load = [&](int st, int slot) __attribute__((always_inline)) {
        const int p = min(8 * st, NP - 8); 
        const uint8_t* b = ub + (uint32_t)p * 16u;
        wa[slot] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(b + va));
        wb[slot] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(b + vb));
        constexpr int PG = GROUP >= 32 ? GROUP / 32 : 1;
        const uint32_t g = FMT == F_MX ? p : FMT == F_NV ? 2 * p : 2 * (p / PG);
        __builtin_memcpy(sc[slot].c, us + g + vs, Scales<FMT, GROUP>::BYTES);
        if (FMT == F_INT) __builtin_memcpy(sc[slot].z, uz + (uint32_t)(p / PG) + vz, Scales<FMT, GROUP>::NG);
      };

      v4f acc4 = {0.f, 0.f, 0.f, 0.f};
      float acc[TB] = {};
      uint64_t again = 0;             // lanes that wrote an output that is not finite
      const int total = nu * mine;
      int lcb = cb0, li = 0;          // next load
      auto load_next = [&](int slot) __attribute__((always_inline)) {
        load(wave + MV_WAVES * li, slot);
        if (++li == mine) {
          li = 0;
          if (lcb + 1 < cb0 + nu)
            point(++lcb);
          else
            aside();
        }
      };
      // the first weights behind x; then this wave's part of x has landed once
      // no more than those are in flight
      point(lcb);
      if (mine <= 0) aside();
#pragma unroll
      for (int k = 0; k < MV_DEPTH - 1; ++k) load_next(k);
      // what the steps need of the lane's place is computed from here on, under
      // the loads (opaque, or the compiler moves it in front of them)
      int place = tid;
      asm volatile("" : "+v"(place));
      const int ln = place & 63, n16 = ln & 15, q = ln >> 4;
      // this lane's rows of x in operand order; the zeros stay where they are
      const uint8_t* xl[TB];
      bool xlive[TB];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        const int t = DIAG ? 4 * tb + (n16 >> 2) : min(n16, rows - 1);
        const bool live = !DIAG || ((n16 & 3) == q && t < rows);
        xl[tb] = live ? xs + t * pitch + 128 * q : zero;
        xlive[tb] = live;
      }

      // one step of the product
      auto step = [&](int st, int slot) __attribute__((always_inline)) {
        const int lc = ln >> 3, lp = ln & 7;
        *reinterpret_cast<v4u*>(wbuf + lc * 128 + ((lp ^ wkey(lc)) << 4)) = wa[slot];
        *reinterpret_cast<v4u*>(wbuf + (lc + 8) * 128 + ((lp ^ wkey(lc + 8)) << 4)) = wb[slot];
        __builtin_amdgcn_wave_barrier();
        v4u w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = *reinterpret_cast<const v4u*>(wbuf + n16 * 128 + (((2 * q + h) ^ wkey(n16)) << 4));
        __builtin_amdgcn_wave_barrier();
        const uint8_t* x[TB];   // of this step: 128 bytes, h * 64 + j * 16
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) x[tb] = xl[tb] + (xlive[tb] ? st * (MV_STEP * 2) : 0);
        auto frag = [&](int tb, int at) __attribute__((always_inline)) {
          return *reinterpret_cast<const v4u*>(x[tb] + at);
        };
        if constexpr (FMT == F_MX) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v4u xf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[j] = frag(0, h * 64 + j * 16);
            const float s = e8m0((sc[slot].c[0] >> (8 * h)) & 0xffu);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc4 = mfma(xf[j], fp4_to_bf16(w[h][j], s), acc4);
          }
        } else if constexpr (FMT == F_NV) {
          float s[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc[slot].c[i], false);
            const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)sc[slot].c[i], true);
            s[4 * i] = lo[0], s[4 * i + 1] = lo[1], s[4 * i + 2] = hi[0], s[4 * i + 3] = hi[1];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __builtin_amdgcn_sched_barrier(0);   // one piece's operands at a time
            v4u b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = fp4_to_bf16(w[h][j], 1.0f);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              v4u xf[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) xf[j] = frag(tb, h * 64 + j * 16);
#pragma unroll
              for (int g = 0; g < 2; ++g) {   // 16 K: two instructions
                v4f p = {0.f, 0.f, 0.f, 0.f};
                p = mfma(xf[2 * g], b[2 * g], p);
                p = mfma(xf[2 * g + 1], b[2 * g + 1], p);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[tb] = fmaf(s[4 * i + 2 * h + g], p[i], acc[tb]);
              }
            }
          }
        } else {
          constexpr int NG = MV_STEP / GROUP, PG = 8 / NG;   // groups, pieces of a group
          float s[NG], z[NG];
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            s[i] = __uint_as_float((i & 1) ? sc[slot].c[i >> 1] & 0xffff0000u : sc[slot].c[i >> 1] << 16);
            z[i] = Ze ? -16.f - (float)((sc[slot].z[i >> 2] >> (8 * (i & 3))) & 0xffu) : -24.f;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            __builtin_amdgcn_sched_barrier(0);   // one piece's operands at a time
            v4u b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = int4_to_bf16(w[h][j], nib, one16);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              // the result's rows are (token 4 tb + q, piece 2i + h)
              const float* sx = xsum + min(4 * tb + q, rows - 1) * steps * 8 + st * 8 + h;
              v4u xf[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) xf[j] = frag(tb, h * 64 + j * 16);
              v4f p;
#pragma unroll
              for (int i = 0; i < 4; ++i) p[i] = z[(2 * i + h) / PG] * sx[2 * i];
#pragma unroll
              for (int j = 0; j < 4; ++j) p = mfma(xf[j], b[j], p);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[tb] = fmaf(s[(2 * i + h) / PG], p[i], acc[tb]);
            }
          }
        }
      };
      // end of a unit: the waves' sums join, bf16 results leave
      auto finish = [&](int cb) __attribute__((always_inline)) {
        float* rd = red + parity * MV_WAVES * rows_max * 16;
        parity ^= 1;
        if constexpr (FMT == F_MX) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * q + i < rows) rd[(wave * rows_max + 4 * q + i) * 16 + n16] = acc4[i];
          acc4 = v4f{0.f, 0.f, 0.f, 0.f};
        } else {
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) {
            if (4 * tb + q < rows) rd[(wave * rows_max + 4 * tb + q) * 16 + n16] = acc[tb];
            acc[tb] = 0.f;
          }
        }
        lds_barrier();
        const int t = place >> 4, n = cb * 16 + (place & 15);
        uint16_t out = 0;
        if (t < rows && n < a.N) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < MV_WAVES; ++w) v += rd[(w * rows_max + t) * 16 + (place & 15)];
          out = __builtin_bit_cast(uint16_t, (__bf16)(v * gs));
          a.y[(size_t)slots[t] * a.N + n] = out;
        }
        again |= __ballot(not_finite(out));
      };

      wait_loads<3 * (MV_DEPTH - 1)>();
      if constexpr (FMT == F_INT) x_finish();
      lds_barrier();

      if (mine == 0) {
        for (int c = 0; c < nu; ++c) finish(cb0 + c);
      } else {
        int cb = cb0, si = 0;
        for (int t = 0; t < total; t += MV_DEPTH) {
#pragma unroll
          for (int k = 0; k < MV_DEPTH; ++k) {
            // loads in every turn, so that each wait is one constant
            load_next((k + MV_DEPTH - 1) % MV_DEPTH);
            if (t + k < total) {
              step(wave + MV_WAVES * si, k);
              if (++si == mine) {
                si = 0;
                finish(cb++);
              }
            }
          }
        }
      }

      // outputs that are not finite once more, each by the whole wave (a lane
      // reads back what it wrote itself); a row of x with a NaN has its NaN
      // already.  8 slots of 8 experts 4096 x 6144 with an infinity in x: 0.5 ms.
      if (__builtin_expect(again != 0, 0)) {
        uint32_t nan_rows = 0;
        for (int r = 0; r < rows; ++r) {
          const uint16_t* xr = a.x + (size_t)((slots[r] * a.per_row_inv) >> 16) * a.K;
          bool nan = false;
          for (int c = ln; c < a.K / 2; c += 64) {
            const uint32_t v = reinterpret_cast<const uint32_t*>(xr)[c];
            nan |= (v & 0x7fffu) > 0x7f80u || (v & 0x7fff0000u) > 0x7f800000u;
          }
          nan_rows |= (__ballot(nan) ? 1u : 0u) << r;
        }
        for (int c = cb0; c < cb0 + nu; ++c) {
          const int t = place >> 4, n = c * 16 + (place & 15);
          const bool live = t < rows && n < a.N && !((nan_rows >> (t & 31)) & 1u);
          uint64_t todo = __ballot(live && not_finite(a.y[(size_t)slots[t] * a.N + n]));
          for (; todo; todo &= todo - 1) {
            const int b = __ffsll((unsigned long long)todo) - 1;
            const int slot = __builtin_amdgcn_readfirstlane(slots[(wave * 64 + b) >> 4]), col = c * 16 + (b & 15);
            const uint16_t* xr = a.x + (size_t)((slot * a.per_row_inv) >> 16) * a.K;
            const float v = exact_output<FMT>(a, (size_t)e * a.N + col, xr, gs);
            if (ln == b) a.y[(size_t)slot * a.N + col] = __builtin_bit_cast(uint16_t, (__bf16)v);
          }
        }
      }
    }
  }
}

constexpr int MV_LDS = 160 * 1024;   // of a CU

template <int FMT, int GROUP, int TB, int WAVES>
hipError_t launch_path(const MatvecArgs& a, int rows, int grid, int lds, hipStream_t stream) {
  if (lds > 64 * 1024) {
    // Past what a launch may have without asking: the kernel may have all of a
    // CU's LDS from its first such call on a device on.  One amount for every
    // call, so that no host thread lowers it between another's request and launch.
    static std::atomic<uint64_t> allowed{0};   // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(&matvec_kernel<FMT, GROUP, TB, WAVES>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, MV_LDS);
      if (e != hipSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_release);
    }
  }
  hipLaunchKernelGGL((matvec_kernel<FMT, GROUP, TB, WAVES>), dim3(grid), dim3(64 * WAVES), lds, stream, a, rows);
  return hipGetLastError();
}

template <int FMT, int GROUP, int WAVES>
hipError_t launch_sets(const MatvecArgs& a, int rows, int grid, int lds, hipStream_t stream) {
  if (FMT == F_MX || rows <= 4) return launch_path<FMT, GROUP, 1, WAVES>(a, rows, grid, lds, stream);
  if (rows <= 8) return launch_path<FMT, GROUP, FMT == F_MX ? 1 : 2, WAVES>(a, rows, grid, lds, stream);
  return launch_path<FMT, GROUP, FMT == F_MX ? 1 : 4, WAVES>(a, rows, grid, lds, stream);
}

template <int WAVES>
hipError_t launch_waves(const MatvecArgs& a, int cus, int64_t units, hipStream_t stream) {
  // rows of an item: all of a dense call's, twice the mean of an expert's (at
  // least four), as far as the LDS holds them; then as many workgroups per CU
  // as there are units, registers and LDS for (and one per slot at least: an
  // item has a slot)
  const int steps = (a.K + MV_STEP - 1) / MV_STEP;
  int rows = std::min(std::min(a.S, 16), a.ids ? std::max(4, 2 * ((a.S + a.E - 1) / a.E)) : 16);
  int per_cu = (int)std::min<int64_t>(mv_per_cu(WAVES, a.fmt != F_MX && rows > 8 ? 4 : 1),
                                      std::max<int64_t>(1, (units + cus - 1) / cus));
  while (per_cu > 1 && mv_lds_bytes(WAVES, steps, std::min(rows, 4)) > MV_LDS / per_cu) --per_cu;
  while (rows > 1 && mv_lds_bytes(WAVES, steps, rows) > MV_LDS / per_cu) --rows;
  const int64_t work = units * (a.ids ? 1 : (a.S + rows - 1) / rows);
  const int grid = std::max(a.S, (int)std::min<int64_t>(work, (int64_t)per_cu * cus));
  const int lds = mv_lds_bytes(WAVES, steps, rows);
  if (a.fmt == F_MX) return launch_sets<F_MX, 32, WAVES>(a, rows, grid, lds, stream);
  if (a.fmt == F_NV) return launch_sets<F_NV, 16, WAVES>(a, rows, grid, lds, stream);
  if (a.group == 32) return launch_sets<F_INT, 32, WAVES>(a, rows, grid, lds, stream);
  if (a.group == 64) return launch_sets<F_INT, 64, WAVES>(a, rows, grid, lds, stream);
  return launch_sets<F_INT, 128, WAVES>(a, rows, grid, lds, stream);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, int cus, hipStream_t stream) {
  const int steps = (a.K + MV_STEP - 1) / MV_STEP;
  if (a.K < MV_STEP || mv_lds_bytes(8, steps, 1) > MV_LDS || (int64_t)a.N * (a.K >> 1) >= (int64_t)1 << 32) {
    const dim3 grid((a.N + 3) / 4, a.S), block(256);
    if (a.fmt == F_MX) hipLaunchKernelGGL(matvec_plain_kernel<F_MX>, grid, block, 0, stream, a);
    else if (a.fmt == F_NV) hipLaunchKernelGGL(matvec_plain_kernel<F_NV>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(matvec_plain_kernel<F_INT>, grid, block, 0, stream, a);
    return hipGetLastError();
  }
  // Eight waves where a CU gets one workgroup in any case: not enough units
  // for two (one row of 2048 x 6144, MXFP4: 8.6 against 10.3 us with four, 5
  // rows of 3583 x 6144, INT4: 10.8 against 11.2), or so many rows of x that
  // the LDS holds no second (16 rows of 6144 x 6144: MXFP4 10.4 against 12.9
  // us, INT4 20.3 against 22.0, NVFP4 15.1 against 16.1).  Else four (24 slots
  // of 6144 x 2048: NVFP4 25.8 against 27.4 us, INT4 28.0 against 32.9).
  const int64_t units = (int64_t)std::min(a.S, a.E) * ((a.N + 15) / 16);
  if (units <= cus || (!a.ids && a.S > 8)) return launch_waves<8>(a, cus, units, stream);
  return launch_waves<4>(a, cus, units, stream);
}

}  // namespace w4a8
