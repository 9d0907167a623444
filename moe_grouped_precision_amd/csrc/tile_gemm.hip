// Matrix products grouped by expert, in LDS tiles on the matrix cores, gfx950:
//
//   forward   C[r, n]     = sum_k A[r, k]  W[e, n, k]        bf16 rows, bf16 weights
//   row grad  dA[r, k]    = sum_n dC[r, n] W[e, n, k]
//   weights   dW[e, n, k] = sum_r dC[r, n] A[r, k]           r over the expert's rows
//   4 by 4    C[r, n]     = sum_k A4[r, k] B4[e, n, k]       MXFP4 rows and weights
//
// All four are out[y, x] = sum_z Y(y, z) X(x, z) with fp32 sums; they differ in
// which index lies contiguous.  A step is 64 bytes of z per row of a tile: 32
// bf16 or 128 FP4 values, one 16x16 matrix instruction deep.  An operand whose z
// is contiguous lies in LDS as rows of 64 bytes, 16-byte chunk c of row r at
// place c ^ (r >> 2 & 3): the 16 lanes of a fragment read then cover all banks.
// One whose z are rows of memory (the weights of the row gradient, both
// operands of the weights') lies as it is, 32 rows of z, chunk c of row z at
// place c ^ swz(z), and its fragments are read by the transposing LDS load
// (ds_read_b64_tr_b16: lanes 4j .. 4j+3 of 16 give row j of a 4 x 16 block, lane i
// gets column i), whose 8 rows in flight swz keeps in different banks.
//
// X is the matrix instruction's first operand, so a lane's four results are four
// consecutive x of one y.
#include "w4a8_kernel.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

namespace w4a8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

enum { FWD = 0, ROWS = 1, WEIGHTS = 2, FOUR = 3 };
constexpr int STEP = 64;     // bytes of z per row and step
constexpr int ZROWS = 32;    // rows of z per step of a transposed operand

// What a chunk past the end of z is read from: zeros, so that whatever the
// buffer holds there (another expert's rows, infinities) stays out of the sums.
__device__ const uint4 zero_chunk = {0, 0, 0, 0};

__device__ __forceinline__ void dma16(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(p), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  // own loads landed and own LDS reads done, then the workgroup's
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}

typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// Place of z rows' chunks, an even number so that a pair of chunks (16 columns)
// stays together.
template <int T>
__device__ __forceinline__ int swz(int z) {
  return 2 * ((z & 3) | ((z >> 1) & 4)) & (T / 8 - 1);
}

// Fragment of 16 rows of an operand with contiguous z: lane 16 q + i holds
// 16 bytes, chunk q of row i.
__device__ __forceinline__ v4i frag_rows(uint32_t tile, int blk, int lane) {
  const int i = lane & 15, q = lane >> 4;
  return *(lds_v4i*)(uintptr_t)(tile + (blk * 16 + i) * STEP + ((q ^ (i >> 2)) << 4));
}
// The same of a transposed one of T columns: lane 16 q + i holds z = 8 q .. 8 q + 7 of
// column i.
template <int T>
__device__ __forceinline__ v4i frag_cols(uint32_t tile, int blk, int lane) {
  const int i = lane & 15, q = lane >> 4;
  const int z = 8 * q + (i >> 2), chunk = 2 * blk + ((i >> 1) & 1), in = (i & 1) * 8;
  const uint32_t a0 = tile + z * (T * 2) + ((chunk ^ swz<T>(z)) << 4) + in;
  // z + 4 has the same place: swz looks at bits 0, 1 and 3
  const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)a0));
  const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(uintptr_t)(a0 + 4 * T * 2)));
  return (v4i){(int)lo[0], (int)lo[1], (int)hi[0], (int)hi[1]};
}

struct Place {
  int e, y0, ny, x0, nx;    // expert, tile
  int r0, rows;             // the expert's rows
};

// The tile of workgroup b, false if it has none or the offsets are not those of
// E experts in R rows.  Tiles of an expert go in groups of 8 row tiles, row
// tiles fastest, and each XCD (workgroups go round them) takes one run of them
// all: what its CUs work on at a time then shares rows and weights in its L2.
template <int MODE, int TY, int TX>
__device__ __forceinline__ bool find_tile(const TileArgs& a, int64_t b, Place& p) {
  const int lane = threadIdx.x & 63;
  const int width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N;
  const int nt = (width + TX - 1) / TX;
  const int fixed = MODE == WEIGHTS ? (a.N + TY - 1) / TY : 0;   // row tiles of every expert
  int sum = 0;
  bool bad = false;
  for (int i = lane; i < a.E; i += 64) {
    const int o0 = a.offsets[i], o1 = a.offsets[i + 1];
    bad |= o1 < o0 || (i == 0 && o0 != 0) || (i == a.E - 1 && o1 > a.R);
    sum += MODE == WEIGHTS ? fixed : (int)((uint32_t)(o1 - o0 + TY - 1) / TY);
  }
  if (__ballot(bad)) return false;
  const int64_t total = (int64_t)__builtin_amdgcn_readlane(wave_inclusive_sum(sum), 63) * nt;
  const int64_t per = (total + 7) >> 3, t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= total) return false;
  int m = (int)(t / nt);   // row tiles before the expert's are whole rows of nt tiles
  int e = 0, mine = fixed;
  if (MODE == WEIGHTS) {
    e = m / fixed;
    m = e * fixed;
  } else {
    int before = 0;
    for (int base = 0;; base += 64) {
      const int i = base + lane;
      const int n = i < a.E ? (a.offsets[i + 1] - a.offsets[i] + TY - 1) / TY : 0;
      const int upto = before + wave_inclusive_sum(n);
      const uint64_t hit = __ballot(m < upto);   // m < total: some lane has it
      if (hit) {
        const int l = __ffsll((unsigned long long)hit) - 1;
        e = base + l;
        mine = __builtin_amdgcn_readlane(n, l);
        m = __builtin_amdgcn_readlane(upto, l) - mine;
        break;
      }
      before = __builtin_amdgcn_readlane(upto, 63);
    }
  }
  const int l = (int)(t - (int64_t)m * nt);
  const int g = l / (8 * nt), rest = l - g * 8 * nt, gm = min(8, mine - 8 * g);
  const int yt = 8 * g + rest % gm, xt = rest / gm;
  p.e = uniform(e);
  p.r0 = uniform(a.offsets[p.e]);
  p.rows = uniform(a.offsets[p.e + 1]) - p.r0;
  p.y0 = uniform(yt) * TY;
  p.ny = min(TY, (MODE == WEIGHTS ? a.N : p.rows) - p.y0);
  p.x0 = uniform(xt) * TX;
  p.nx = min(TX, width - p.x0);
  return true;
}

// 16 bytes of a row at any 2-byte alignment; n < 8 values from its end one by
// one, none past it.
__device__ __forceinline__ v4i load_any(const uint8_t* p, int n) {
  v4i v = {0, 0, 0, 0};
  if (n >= 8) {
    __builtin_memcpy(&v, p, 16);
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) v[i >> 1] |= (int)((uint32_t)q[i] << (16 * (i & 1)));
  }
  return v;
}

// TY x TX tiles, WY x WX waves, NS steps of the operands in LDS.  DIRECT: rows
// are whole 16-byte chunks at 16-byte addresses and go straight to LDS;
// otherwise through registers.
template <int MODE, int TY, int TX, int WY, int WX, int NS, bool DIRECT, typename OUT>
struct Tile {
  static constexpr bool YT = MODE == WEIGHTS, XT = MODE == WEIGHTS || MODE == ROWS;   // transposed operands
  static constexpr int NW = WY * WX, THREADS = 64 * NW;
  static constexpr int MY = TY / WY / 16, MX = TX / WX / 16;
  static constexpr int IY = TY / 16 / NW, IX = TX / 16 / NW, NI = IY + IX;   // loads of 1 KB per wave and step
  static constexpr int SCALES = MODE == FOUR ? (TY + TX) * 4 : 0;
  static constexpr int SY = MODE == FOUR ? (TY / 64 + NW - 1) / NW : 0, SX = MODE == FOUR ? (TX / 64 + NW - 1) / NW : 0;
  static constexpr int STAGE = (TY + TX) * STEP + SCALES;
  static constexpr int LDS = STAGE * NS;
  static constexpr int PER = NI + SY + SX;
  static_assert(TY / 16 % NW == 0 && TX / 16 % NW == 0, "whole loads per wave");
  static_assert(DIRECT || MODE != FOUR, "FP4 rows are whole chunks");

  // This wave's i-th load of a step: its place in the tile and the lane's chunk.
  template <int T, bool TR>
  static __device__ __forceinline__ void chunk_of(int j, int lane, int& row, int& chunk) {
    if (TR) {
      constexpr int CPR = T / 8;
      row = j * (64 / CPR) + lane / CPR;                // z
      chunk = (lane % CPR) ^ swz<T>(row);               // of 8 columns
    } else {
      row = j * 16 + (lane >> 2);
      chunk = (lane & 3) ^ ((lane >> 4) & 3);           // of z
    }
  }

  static __device__ __forceinline__ void run(const TileArgs& a, int64_t b) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t lds = lds_u32(smem);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    Place p;
    if (!find_tile<MODE, TY, TX>(a, b, p)) return;

    // operands: base of the tile, bytes from row to row, extent of z
    const int zn = MODE == WEIGHTS ? p.rows : MODE == ROWS ? a.N : a.K;
    const int ybytes = MODE == FOUR ? a.K / 2 : MODE == FWD ? a.K * 2 : a.N * 2;
    const int xbytes = MODE == FOUR ? a.K / 2 : a.K * 2;
    const uint8_t* Y = a.Y + (size_t)(p.r0 + (MODE == WEIGHTS ? 0 : p.y0)) * ybytes + (MODE == WEIGHTS ? p.y0 * 2 : 0);
    const uint8_t* X = MODE == WEIGHTS ? a.X + (size_t)p.r0 * xbytes + p.x0 * 2
                       : MODE == ROWS  ? a.X + (size_t)p.e * a.N * xbytes + p.x0 * 2
                                       : a.X + ((size_t)p.e * a.N + p.x0) * xbytes;
    const int steps = MODE == FOUR ? zn / 128 : (zn + 31) / 32;
    const int full = MODE == FOUR ? steps : zn / 32;   // steps without an end of z in them

    v4f acc[MY][MX];
#pragma unroll
    for (int i = 0; i < MY; ++i)
#pragma unroll
      for (int j = 0; j < MX; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

    // the lane's chunks of a step
    const uint8_t* src[NI];
    int left[NI];     // values of z (or, transposed, rows of z) from the chunk on to the end of z
    int wide[NI];     // columns of a transposed chunk inside the tile's extent
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool isy = i < IY;
      const int j = wave + NW * (isy ? i : i - IY);
      int row, chunk;
      if (isy) chunk_of<TY, YT>(j, lane, row, chunk);
      else chunk_of<TX, XT>(j, lane, row, chunk);
      const int extent = isy ? p.ny : p.nx, pitch = isy ? ybytes : xbytes;
      const uint8_t* base = isy ? Y : X;
      if (isy ? YT : XT) {
        wide[i] = DIRECT ? 8 : max(0, min(8, extent - chunk * 8));
        const int c = DIRECT ? min(chunk * 8, extent - 8) : chunk * 8;   // past the end: any column, never stored
        src[i] = base + (size_t)row * pitch + (DIRECT || wide[i] > 0 ? c * 2 : 0);
        left[i] = zn - row;
      } else {
        wide[i] = 8;
        src[i] = base + (size_t)min(row, extent - 1) * pitch + chunk * 16;
        left[i] = zn - chunk * 8;
      }
    }
    const size_t ystep = YT ? (size_t)ZROWS * ybytes : STEP, xstep = XT ? (size_t)ZROWS * xbytes : STEP;

    // FP4: the E8M0 codes of a step, 4 per row
    const uint8_t* ssrc[SY + SX + 1];
    uint32_t sdst[SY + SX + 1];
    if constexpr (MODE == FOUR) {
      const int g = a.K / 32;
#pragma unroll
      for (int i = 0; i < SY + SX; ++i) {
        const bool isy = i < SY;
        const int blocks = (isy ? TY : TX) / 64, blk = (wave + NW * (isy ? i : i - SY)) % blocks;
        const int row = min(blk * 64 + lane, (isy ? p.ny : p.nx) - 1);
        ssrc[i] = isy ? a.SY + (size_t)(p.r0 + p.y0 + row) * g : a.SX + ((size_t)p.e * a.N + p.x0 + row) * g;
        sdst[i] = (TY + TX) * STEP + (isy ? 0 : TY * 4) + blk * 256;
      }
    }

    auto place = [&](int i, uint32_t stage) {
      return stage + (i < IY ? (wave + NW * i) * 1024 : TY * STEP + (wave + NW * (i - IY)) * 1024);
    };
    auto issue = [&](int s, uint32_t stage) {   // DIRECT: the loads of step s
      const bool whole = s < full;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint8_t* q = src[i];
        if (!whole && left[i] - 32 * s <= 0) q = reinterpret_cast<const uint8_t*>(&zero_chunk);
        dma16(q, place(i, stage));
        src[i] += i < IY ? ystep : xstep;
      }
      if constexpr (MODE == FOUR) {
#pragma unroll
        for (int i = 0; i < SY + SX; ++i) {
          vm_dma4(ssrc[i], stage + sdst[i]);
          ssrc[i] += 4;
        }
      }
    };

    const int wy = wave / WX, wx = wave % WX;
    auto compute = [&](uint32_t stage) {
      v4i fy[MY], fx[MX];
#pragma unroll
      for (int i = 0; i < MY; ++i)
        fy[i] = YT ? frag_cols<TY>(stage, wy * MY + i, lane) : frag_rows(stage, wy * MY + i, lane);
#pragma unroll
      for (int j = 0; j < MX; ++j)
        fx[j] = XT ? frag_cols<TX>(stage + TY * STEP, wx * MX + j, lane) : frag_rows(stage + TY * STEP, wx * MX + j, lane);
      if constexpr (MODE == FOUR) {
        int ey[MY], ex[MX];
        const uint32_t sc = stage + (TY + TX) * STEP + (lane & 15) * 4 + (lane >> 4);
#pragma unroll
        for (int i = 0; i < MY; ++i) ey[i] = *(lds_u8*)(uintptr_t)(sc + (wy * MY + i) * 64);
#pragma unroll
        for (int j = 0; j < MX; ++j) ex[j] = *(lds_u8*)(uintptr_t)(sc + TY * 4 + (wx * MX + j) * 64);
#pragma unroll
        for (int i = 0; i < MY; ++i)
#pragma unroll
          for (int j = 0; j < MX; ++j) {
            const v8i x8 = {fx[j][0], fx[j][1], fx[j][2], fx[j][3], 0, 0, 0, 0};
            const v8i y8 = {fy[i][0], fy[i][1], fy[i][2], fy[i][3], 0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x8, y8, acc[i][j], 4, 4, 0, ex[j], 0, ey[i]);
          }
      } else {
#pragma unroll
        for (int i = 0; i < MY; ++i)
#pragma unroll
          for (int j = 0; j < MX; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, fx[j]),
                                                                __builtin_bit_cast(v8bf, fy[i]), acc[i][j], 0, 0, 0);
      }
    };

    if constexpr (DIRECT) {
#pragma unroll
      for (int s = 0; s < NS - 1; ++s)
        if (s < steps) issue(s, lds + s * STAGE);
      uint32_t slot = 0, next = (NS - 1) * STAGE;
      for (int s = 0; s < steps; ++s) {
        // step s landed: the NS - 2 issued after it may still be under way
        if (s + NS - 2 < steps) wait_and_meet<(NS - 2) * PER>();
        else wait_and_meet<0>();
        if (s + NS - 1 < steps) issue(s + NS - 1, lds + next);   // where step s - 1 was
        compute(lds + slot);
        slot = slot == (NS - 1) * STAGE ? 0 : slot + STAGE;
        next = next == (NS - 1) * STAGE ? 0 : next + STAGE;
      }
    } else {
      v4i reg[NI];
      auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const bool tr = i < IY ? YT : XT;
          const int z = left[i] - 32 * s;
          reg[i] = load_any(src[i], z <= 0 ? 0 : tr ? wide[i] : z);
          src[i] += i < IY ? ystep : xstep;
        }
      };
      auto put = [&](uint32_t stage) {
#pragma unroll
        for (int i = 0; i < NI; ++i) *(lds_v4i*)(uintptr_t)(place(i, stage) + lane * 16) = reg[i];
      };
      if (steps > 0) {
        fetch(0);
        put(lds);
        __syncthreads();
      }
      for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) fetch(s + 1);
        compute(lds + (s & 1) * STAGE);
        if (s + 1 < steps) put(lds + ((s + 1) & 1) * STAGE);
        __syncthreads();
      }
    }

    if (MODE == WEIGHTS && a.accumulate && steps == 0) return;
    const int width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N;
    OUT* out = static_cast<OUT*>(a.out) +
               (MODE == WEIGHTS ? (size_t)p.e * a.N + p.y0 : (size_t)(p.r0 + p.y0)) * width + p.x0;
#pragma unroll
    for (int i = 0; i < MY; ++i) {
      const int y = (wy * MY + i) * 16 + (lane & 15);
#pragma unroll
      for (int j = 0; j < MX; ++j) {
        const int x = (wx * MX + j) * 16 + 4 * (lane >> 4);
        if (y >= p.ny || x >= p.nx) continue;
        OUT* o = out + (size_t)y * width + x;
        v4f v = acc[i][j];
        const int n = DIRECT ? 4 : min(4, p.nx - x);
        if (MODE == WEIGHTS && a.accumulate) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < n) v[c] += sizeof(OUT) == 4 ? (float)o[c] : __uint_as_float((uint32_t)(uint16_t)o[c] << 16);
        }
        if constexpr (sizeof(OUT) == 4) {
          if (DIRECT) *reinterpret_cast<v4f*>(o) = v;
          else
            for (int c = 0; c < n; ++c) o[c] = v[c];
        } else {
          if (DIRECT) store_bf16x4(o, v);
          else
            for (int c = 0; c < n; ++c) o[c] = __builtin_bit_cast(uint16_t, (__bf16)v[c]);
        }
      }
    }
  }
};

template <int MODE, int TY, int TX, int WY, int WX, int NS, bool DIRECT, typename OUT>
__global__ void __launch_bounds__(64 * WY * WX, 2)
tile_kernel(TileArgs a, int64_t b0) {
  Tile<MODE, TY, TX, WY, WX, NS, DIRECT, OUT>::run(a, b0 + blockIdx.x);
}

template <int MODE, int TY, int TX, int WY, int WX, int NS, bool DIRECT, typename OUT>
hipError_t launch(const TileArgs& a, hipStream_t stream) {
  using T = Tile<MODE, TY, TX, WY, WX, NS, DIRECT, OUT>;
  const auto kernel = &tile_kernel<MODE, TY, TX, WY, WX, NS, DIRECT, OUT>;
  if (T::LDS > 64 * 1024) {
    // more than a launch has without asking; once per device
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
      if (e != hipSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_release);
    }
  }
  // tiles: known for the weights, otherwise at most (each expert's last may be
  // part of one); workgroups come in eights, one per XCD
  const int64_t width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N, nt = (width + TX - 1) / TX;
  const int64_t rows = MODE == WEIGHTS ? (int64_t)a.E * ((a.N + TY - 1) / TY)
                                       : (a.R + (int64_t)std::min(a.E, a.R) * (TY - 1)) / TY;
  return in_launches((rows * nt + 7) / 8 * 8, T::THREADS, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL((tile_kernel<MODE, TY, TX, WY, WX, NS, DIRECT, OUT>), dim3((unsigned)n), dim3(T::THREADS), T::LDS,
                       stream, a, b);
  });
}

bool chunks16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int MODE, typename OUT>
hipError_t launch_bf16(const TileArgs& a, hipStream_t stream) {
  if (a.N % 8 || a.K % 8 || !chunks16(a.Y) || !chunks16(a.X) || !chunks16(a.out))
    return launch<MODE, 128, 128, 2, 2, 2, false, OUT>(a, stream);
  return launch<MODE, 128, 256, 2, 2, 3, true, OUT>(a, stream);
}

}  // namespace

hipError_t launch_grouped_bf16(const TileArgs& a, hipStream_t stream) { return launch_bf16<FWD, uint16_t>(a, stream); }
hipError_t launch_grouped_dgrad(const TileArgs& a, hipStream_t stream) { return launch_bf16<ROWS, uint16_t>(a, stream); }
hipError_t launch_grouped_wgrad(const TileArgs& a, bool f32, hipStream_t stream) {
  return f32 ? launch_bf16<WEIGHTS, float>(a, stream) : launch_bf16<WEIGHTS, uint16_t>(a, stream);
}
hipError_t launch_grouped_a4(const TileArgs& a, hipStream_t stream) {
  return launch<FOUR, 128, 256, 2, 2, 3, true, uint16_t>(a, stream);
}

}  // namespace w4a8
