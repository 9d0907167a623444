// Matrix products grouped by expert, in LDS tiles on the matrix cores, gfx950:
//
//   forward   C[r, n]     = sum_k A[r, k]  W[e, n, k]        bf16 rows, bf16 weights
//   row grad  dA[r, k]    = sum_n dC[r, n] W[e, n, k]
//   weights   dW[e, n, k] = sum_r dC[r, n] A[r, k]           r over the expert's rows
//   4 by 4    C[r, n]     = sum_k A4[r, k] B4[e, n, k]       MXFP4 rows and weights
//
// All four are out[y, x] = sum_z Y(y, z) X(x, z) with fp32 sums; they differ in
// which index lies contiguous.  A step is 64 KS bytes of z per row of a tile: 32 KS
// bf16 or 128 KS FP4 values, KS 16x16 matrix instructions deep.  An operand whose z
// is contiguous lies in LDS as rows of a step's bytes, 16-byte chunk c of row r at
// place c ^ key(r), so that a fragment read covers all banks.  One whose z are rows
// of memory (the weights of the row gradient, both operands of the weights') lies
// as it is, 32 KS rows of z, chunk c of row z at place c ^ swz(z), and its fragments
// are read by the transposing LDS load (ds_read_b64_tr_b16: lanes 4j .. 4j+3 of 16
// give row j of a 4 x 16 block, lane i gets column i), whose 8 rows in flight swz
// keeps in different banks.
//
// What bounds them (32 experts 4096 x 6144, unevenly filled).  The forward product
// of 9216 rows, 575 us, 1.8 GB: its loads.  They alone take as long; a CU has 80 lines
// on their way at a mean latency of 505 cycles, 6.2 GB come from L2 and 2.1 of them
// from memory, the matrix cores are 0.4 busy.  The row gradient, 1.65 TFLOP in 1517 us,
// and the weights', 3.3 in 2839 (2560 without its 1.6 GB of stores): the matrix cores
// 0.50 and 0.58 busy at 2.0 and 1.9 GHz, where normal values alone keep them at 2070
// TFLOP/s; half the misses in L2 do not change it.  4 by 4 bits, 6.6 in 1875: LDS, whose
// reads take as long as the matrix instructions, and the stores.  Few rows: the
// weights' bytes, 4.9 TB/s.
// Tried on the forward product and the weights' gradient, us: loads in one burst 728
// and 5020; steps of 64 bytes (half lines) in 4 or 5 stages 735, 2774; 128 x 256 in
// two stages 751, 256 x 256 in two 637, 192 x 192 in three 620 (605 on that day);
// 32x32x16 instructions 647, 2992; 4 waves of 128 x 128 800, 3267; loads to L2 ahead
// 740; nontemporal loads 1018; workgroups that stay and load the next tile's first
// steps before they store 613 (617 on that day).
//
// X is the matrix instruction's first operand, so a lane's four results are four
// consecutive x of one y.
#include "tile_place.h"
#include "w4a8_kernel.h"
#include "w4a8_launch.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace w4a8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

enum { FWD = PRODUCT_FWD, ROWS = PRODUCT_ROWS, WEIGHTS = PRODUCT_WEIGHTS, FOUR = PRODUCT_FOUR };
constexpr int FEW_ROWS = 48, MANY_ROWS = 768;   // of an expert in the mean: see tile_of
constexpr int64_t CUS = 256;   // of an MI355X; only speed depends on it

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

// Place of the chunks of a row with contiguous z.  A 16-byte read of a wave is
// served in passes of 16 lanes over all banks, lanes 0-3, 12-15, 20-27 and the
// others of each half; these keys put 16 different places in each.
template <int KS>
__device__ __forceinline__ int key(int row) {
  return KS == 1 ? -(row >> 2) & 3 : (row >> 1) & 7;
}
// Fragment h of row block blk of an operand whose tile lies at `tile`: lane 16 q +
// i holds 16 bytes, chunk 4 h + q of row i.  (A pointer and a constant, so that
// the block goes into the instruction's offset.)
template <int KS>
__device__ __forceinline__ uint32_t rows_base(uint32_t tile, int h, int lane) {
  const int i = lane & 15, q = lane >> 4;
  return tile + i * (64 * KS) + (((4 * h + q) ^ key<KS>(i)) << 4);
}
template <int KS>
__device__ __forceinline__ v4i frag_rows(uint32_t base, int blk) {
  return *(lds_v4i*)((lds_u8*)(uintptr_t)base + blk * 16 * (64 * KS));
}
// The same of a transposed one of T columns: lane 16 q + i holds z = 32 h + 8 q ..
// 8 q + 7 of column i.  The block's low bits meet swz's in the chunk's number.
template <int T>
__device__ __forceinline__ uint32_t cols_base(int lane) {   // of a tile at 0, block 0
  const int i = lane & 15, q = lane >> 4, z = 8 * q + (i >> 2);
  return z * (T * 2) + ((((i >> 1) & 1) ^ swz<T>(z)) << 4) + (i & 1) * 8;
}
template <int T>
__device__ __forceinline__ v4i frag_cols(uint32_t base, uint32_t tile, int blk, int h) {
  constexpr int LOW = T / 16 < 8 ? T / 16 - 1 : 7;
  lds_u8* p = (lds_u8*)(uintptr_t)(tile + (base ^ ((blk & LOW) << 5))) + (blk & ~LOW) * 32 + h * 32 * (T * 2);
  // z + 4 has the same place: swz looks at bits 0, 1 and 3
  const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p));
  const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * T * 2)));
  return (v4i){(int)lo[0], (int)lo[1], (int)hi[0], (int)hi[1]};
}

struct Place {
  int e, y0, ny, x0, nx;    // expert, tile
  int r0, rows;             // the expert's rows
  int odd;                  // the tiles as a chessboard
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
    if (MODE != WEIGHTS) sum += pieces_of(o1 - o0, TY);   // of no use where bad
  }
  if (__ballot(bad)) return false;
  int64_t t;
  int m = 0, e = 0, mine = fixed;
  if (MODE == WEIGHTS) {
    // a tile costs what its expert has rows: every XCD gets an eighth of each
    // expert, the first one another XCD each time (it may be all there is)
    const int all = fixed * nt, per = (all + 7) >> 3;
    const int64_t j = b >> 3;
    e = (int)(j / per);
    t = ((b + e + blockIdx.y) & 7) * per + (j - (int64_t)e * per);
    if (e >= a.E || t >= all) return false;
  } else {
    const int64_t total = (int64_t)__builtin_amdgcn_readlane(wave_inclusive_sum(sum), 63) * nt;
    const int64_t per = (total + 7) >> 3;
    t = ((b + blockIdx.y) & 7) * per + (b >> 3);
    if ((b >> 3) >= per || t >= total) return false;
    m = (int)(t / nt);   // row tiles before the expert's are whole rows of nt tiles
    int before = 0;
    for (int base = 0;; base += 64) {
      const int i = base + lane;
      const int n = i < a.E ? pieces_of(a.offsets[i + 1] - a.offsets[i], TY) : 0;
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
  if (MODE == WEIGHTS) {
    p.y0 = uniform(yt) * TY;
    p.ny = min(TY, a.N - p.y0);
  } else {
    // an expert's rows in equal tiles of whole blocks of 16: the kernel leaves
    // out blocks that a tile does not have
    const int per = rows_per_tile(p.rows, mine);
    p.y0 = uniform(yt * per);
    p.ny = uniform(min(per, p.rows - p.y0));
  }
  p.odd = uniform((yt ^ xt) & 1);
  p.x0 = uniform(xt) * TX;
  p.nx = min(TX, width - p.x0);
  return true;
}

// 16 bytes of a row at any 2-byte alignment, n of its 8 values.  The last ones of
// a row are the row's last 16 bytes, moved down by `only` when they are used: a
// load under a condition has to be waited for where the condition ends.
__device__ __forceinline__ v4i load_any(const uint8_t* p, int n) {
  v4i v;
  const uint8_t* q = n <= 0 ? reinterpret_cast<const uint8_t*>(&zero_chunk) : p - 2 * (8 - min(n, 8));
  __builtin_memcpy(&v, q, 16);
  return v;
}
__device__ __forceinline__ v4i only(v4i v, int n) {
  const int by = n <= 0 || n >= 8 ? 0 : 8 - n;
  if (by & 4) v = (v4i){v[2], v[3], 0, 0};
  if (by & 2) v = (v4i){v[1], v[2], v[3], 0};
  if (by & 1)
    v = (v4i){(int)__builtin_amdgcn_alignbit(v[1], v[0], 16), (int)__builtin_amdgcn_alignbit(v[2], v[1], 16),
              (int)__builtin_amdgcn_alignbit(v[3], v[2], 16), (int)((uint32_t)v[3] >> 16)};
  return v;
}
// Rows of fewer than 8 values, one by one.
__device__ __forceinline__ v4i load_few(const uint8_t* p, int n) {
  v4i v = {0, 0, 0, 0};
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) v[i >> 1] |= (int)((uint32_t)q[i] << (16 * (i & 1)));
  return v;
}

// A lane's 16 bytes of load j (1 KB of LDS, so 64 KS bytes of 16 / KS rows or T columns
// of rows of z) of an operand: its row, or row of z, and its chunk.
template <int T, bool TR, int KS>
__device__ __forceinline__ void chunk_of(int j, int lane, int& row, int& chunk) {
  constexpr int CPR = TR ? T / 8 : 4 * KS;
  row = j * (64 / CPR) + lane / CPR;
  chunk = (lane % CPR) ^ (TR ? swz<T>(row) : key<KS>(row & 15));
}

// What the kernels of one product have in common.  With a.slices > 1 a workgroup
// takes one slice of z (blockIdx.y, whole steps), into an array of its own.
template <int MODE>
struct Operands {
  static constexpr bool YT = MODE == WEIGHTS, XT = MODE == WEIGHTS || MODE == ROWS;   // transposed operands
  const uint8_t *Y, *X;   // of the tile, at the first z
  int ybytes, xbytes;     // from row to row
  int zn;                 // extent of z
  int width;              // of the output
  size_t out0;            // the slice's array
  __device__ __forceinline__ Operands(const TileArgs& a, const Place& p) {
    zn = MODE == WEIGHTS ? p.rows : MODE == ROWS ? a.N : a.K;
    ybytes = MODE == FOUR ? a.K / 2 : MODE == FWD ? a.K * 2 : a.N * 2;
    xbytes = MODE == FOUR ? a.K / 2 : a.K * 2;
    width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N;
    Y = a.Y + (size_t)(p.r0 + (MODE == WEIGHTS ? 0 : p.y0)) * ybytes + (MODE == WEIGHTS ? p.y0 * 2 : 0);
    X = MODE == WEIGHTS ? a.X + (size_t)p.r0 * xbytes + p.x0 * 2
        : MODE == ROWS  ? a.X + (size_t)p.e * a.N * xbytes + p.x0 * 2
                        : a.X + ((size_t)p.e * a.N + p.x0) * xbytes;
    out0 = 0;
    if (a.slices > 1) {
      const int each = slice_of(zn, a.slices, MODE == FOUR ? 512 : 64), z0 = min(zn, (int)blockIdx.y * each);
      zn = min(zn - z0, each);
      Y += YT ? (size_t)z0 * ybytes : MODE == FOUR ? z0 / 2 : z0 * 2;
      X += XT ? (size_t)z0 * xbytes : MODE == FOUR ? z0 / 2 : z0 * 2;
      out0 = (size_t)blockIdx.y * (MODE == WEIGHTS ? (size_t)a.E * a.N : (size_t)a.R) * width;
    }
  }
};

// Four of the lane's results added to a bf16 out[y][x .. x+3], with one rounding
// (131072 rows, 32 experts 6144 x 2048: 3220 us, 2621 into a new array; fp32, in
// whole lines, 3084 and 2766).
template <int MODE>
__device__ __forceinline__ void add_to(const TileArgs& a, const Place& p, const Operands<MODE>& op, int y, int x, v4f v) {
  if (y >= p.ny || x >= p.nx) return;
  uint16_t* o = static_cast<uint16_t*>(a.out) + ((size_t)p.e * a.N + p.y0 + y) * op.width + p.x0 + x;
  const int n = min(4, p.nx - x);
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (c < n) v[c] += __uint_as_float((uint32_t)o[c] << 16);
  if (a.wide) {
    store_bf16x4(o, v);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < n) o[c] = __builtin_bit_cast(uint16_t, (__bf16)v[c]);
  }
}

// Lanes 8 .. 15 of every 16 of a with lanes 0 .. 7 of b.
__device__ __forceinline__ void swap_halves(v4i& a, v4i& b) {
  const v4i t = a;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    a[c] = __builtin_amdgcn_update_dpp(a[c], b[c], 0x128, 0xf, 0xc, false);   // row_ror:8
    b[c] = __builtin_amdgcn_update_dpp(b[c], t[c], 0x128, 0xf, 0x3, false);
  }
}

// The lane's results of a row block, MX column blocks from x on, to memory.  In the
// instruction's layout a store has 32 (bf16) or 64 bytes of each of 16 rows, and the
// tiles of a round all store at a time, while nothing else runs on their CUs: lanes
// exchange values until a store has whole lines, and these pass the L2 cache that
// the next tiles' operands lie in.  131072 rows, 4 by 4 bits, 1990 us, so 1909 and
// past the cache 1875 (without any store 1670); weights' gradient 2879, 2866, 2839;
// row gradient 1564, 1528, 1517; forward 597, 590, 579.  What reads the output next
// takes 5% longer to 16% less.
template <int MODE, int MX, typename OUT>
__device__ __forceinline__ void put_block(const TileArgs& a, const Place& p, const Operands<MODE>& op, int y, int x,
                                          const v4f (&acc)[MX]) {
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  if (sizeof(OUT) == 2 && MODE == WEIGHTS && a.accumulate) {
#pragma unroll
    for (int j = 0; j < MX; ++j) add_to<MODE>(a, p, op, y + i, x + 16 * j + 4 * q, acc[j]);
    return;
  }
  constexpr int PER = 16 / sizeof(OUT), PAIRS = MX * 16 / (4 * PER) / 2;   // values of a store, pairs of stores
  auto store = [&](int row, int col, v4i v) {
    if (row >= p.ny || col >= p.nx) return;
    OUT* o = static_cast<OUT*>(a.out) + op.out0 +
             (MODE == WEIGHTS ? (size_t)p.e * a.N + p.y0 + row : (size_t)(p.r0 + p.y0 + row)) * op.width + p.x0 + col;
    if (a.wide) {
      if (sizeof(OUT) == 4 && MODE == WEIGHTS && a.accumulate)
        v = __builtin_bit_cast(v4i, __builtin_bit_cast(v4f, v) + *reinterpret_cast<const v4f*>(o));
      __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(o));
      return;
    }
    // rows at any address: 16 bytes all the same, a row's end value by value
    const int n = min(PER, p.nx - col);
    if (sizeof(OUT) == 4 && MODE == WEIGHTS && a.accumulate) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) v[c] = __float_as_int(__int_as_float(v[c]) + (float)o[c]);
    }
    if (n == PER) {
      __builtin_memcpy(o, &v, 16);
    } else {
#pragma unroll
      for (int c = 0; c < PER - 1; ++c)
        if (c < n) {
          if constexpr (sizeof(OUT) == 4) o[c] = __int_as_float(v[c]);
          else o[c] = (uint16_t)((uint32_t)v[c >> 1] >> (16 * (c & 1)));
        }
    }
  };
  v4i v[MX * 16 / (4 * PER)];
  if constexpr (sizeof(OUT) == 4) {
#pragma unroll
    for (int j = 0; j < MX; ++j) v[j] = __builtin_bit_cast(v4i, acc[j]);
  } else {
    // blocks 2 j and 2 j + 1: a lane gets 8 columns of one, 4 (q & 2) of block q & 1
#pragma unroll
    for (int j = 0; j < MX / 2; ++j)
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const auto pack = [&](v4f f) {
          return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f){f[2 * d], f[2 * d + 1]}, v2bf));
        };
        const auto r = __builtin_amdgcn_permlane16_swap(pack(acc[2 * j]), pack(acc[2 * j + 1]), false, false);
        v[j][d] = (int)r[0];
        v[j][2 + d] = (int)r[1];
      }
  }
  // a store's columns of its first or only 64 bytes of a row
  const int col = sizeof(OUT) == 4 ? x + 4 * q : x + 16 * (q & 1) + 4 * (q & 2);
  if constexpr (PAIRS == 0) {
    store(y + i, col, v[0]);
  } else {
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      swap_halves(v[2 * j], v[2 * j + 1]);
      const int at = col + (2 * j + (i >> 3)) * (4 * PER);
      store(y + (i & 7), at, v[2 * j]);
      store(y + 8 + (i & 7), at, v[2 * j + 1]);
    }
  }
}

__device__ __forceinline__ v4f mfma_bf16(v4i x, v4i y, v4f acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), acc, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Rows that are no whole 16-byte chunks at 16-byte addresses: through registers,
// 128 x 128 tiles, steps of 32 KS z, two of them in LDS and one on its way (a second
// one changes nothing).  Bound by the loads at 2-byte addresses and the writes to LDS.
// ---------------------------------------------------------------------------
template <int MODE, int KS_, typename OUT>
struct General {
  static constexpr int TY = 128, TX = 128, KS = KS_, NW = 4, THREADS = 256, M = 4, NI = TY * KS / 16 / NW, ZSTEP = 32 * KS;
  static constexpr int STAGE = (TY + TX) * 64 * KS, LDS = 2 * STAGE, PER_SIMD = 2;

  static __device__ __forceinline__ void run(const TileArgs& a, int64_t b, uint32_t lds) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    Place p;
    if (!find_tile<MODE, TY, TX>(a, b, p)) return;
    const Operands<MODE> op(a, p);
    constexpr bool YT = Operands<MODE>::YT, XT = Operands<MODE>::XT;
    const int steps = pieces_of(op.zn, ZSTEP);
    v4f acc[M][M];
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < M; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

    // the lane's chunks of a step
    const uint8_t* src[2 * NI];
    int left[2 * NI];   // z from the chunk on to the end
    int wide[2 * NI];   // columns of a transposed chunk inside the tile's extent
#pragma unroll
    for (int i = 0; i < 2 * NI; ++i) {
      const bool isy = i < NI;
      const int j = wave + NW * (i % NI);
      int row, chunk;
      if (isy) chunk_of<TY, YT, KS>(j, lane, row, chunk);
      else chunk_of<TX, XT, KS>(j, lane, row, chunk);
      const int extent = isy ? p.ny : p.nx, pitch = isy ? op.ybytes : op.xbytes;
      const uint8_t* base = isy ? op.Y : op.X;
      if (isy ? YT : XT) {
        wide[i] = max(0, min(8, extent - chunk * 8));
        src[i] = base + (size_t)row * pitch + chunk * 16;
        left[i] = op.zn - row;
      } else {
        wide[i] = 8;
        src[i] = base + (size_t)min(row, extent - 1) * pitch + chunk * 16;
        left[i] = op.zn - chunk * 8;
      }
    }
    const size_t ystep = YT ? (size_t)ZSTEP * op.ybytes : 64 * KS, xstep = XT ? (size_t)ZSTEP * op.xbytes : 64 * KS;
    v4i reg[2 * NI];
    const bool few_y = op.ybytes < 16, few_x = op.xbytes < 16;
    // values of chunk i in step s
    auto values = [&](int i, int s) {
      const int z = left[i] - ZSTEP * s;
      return (i < NI ? YT : XT) ? (z > 0 ? wide[i] : 0) : z;
    };
    auto fetch = [&](int s) {
#pragma unroll
      for (int i = 0; i < 2 * NI; ++i) {
        const int n = values(i, s);
        if (i < NI ? few_y : few_x) reg[i] = load_few(src[i], n);
        else reg[i] = load_any(src[i], n);
        src[i] += i < NI ? ystep : xstep;
      }
    };
    // which operands have such ends, in any step or in the last
    const bool end_y = !few_y && (YT ? (p.ny & 7) != 0 : (op.zn & 7) != 0);
    const bool end_x = !few_x && (XT ? (p.nx & 7) != 0 : (op.zn & 7) != 0);
    auto fill = [&](int s, int to) {
#pragma unroll
      for (int i = 0; i < 2 * NI; ++i) {
        if ((i < NI ? end_y : end_x) && ((i < NI ? YT : XT) || s == steps - 1)) reg[i] = only(reg[i], values(i, s));
        *(lds_v4i*)(uintptr_t)(lds + to * STAGE + (i / NI) * TY * 64 * KS + (wave + NW * (i % NI)) * 1024 + lane * 16) =
            reg[i];
      }
    };
    const int wy = wave >> 1, wx = wave & 1;
    auto step = [&](int s, int at) {
      if (s + 1 < steps) fetch(s + 1);
      const uint32_t stage = lds + at * STAGE;
#pragma unroll
      for (int h = 0; h < KS; ++h) {
        v4i fy[M], fx[M];
#pragma unroll
        for (int i = 0; i < M; ++i) {
          fy[i] = YT ? frag_cols<TY>(cols_base<TY>(lane), stage, wy * M + i, h)
                     : frag_rows<KS>(rows_base<KS>(stage, h, lane), wy * M + i);
          fx[i] = XT ? frag_cols<TX>(cols_base<TX>(lane), stage + TY * 64 * KS, wx * M + i, h)
                     : frag_rows<KS>(rows_base<KS>(stage + TY * 64 * KS, h, lane), wx * M + i);
        }
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
          for (int j = 0; j < M; ++j) acc[i][j] = mfma_bf16(fx[j], fy[i], acc[i][j]);
      }
      if (s + 1 < steps) fill(s + 1, at ^ 1);
      __syncthreads();
    };
    if (steps > 0) {
      fetch(0);
      fill(0, 0);
      __syncthreads();
    }
    for (int s = 0; s < steps; ++s) step(s, s & 1);
    if (MODE == WEIGHTS && a.accumulate && steps == 0) return;
#pragma unroll
    for (int i = 0; i < M; ++i)
      put_block<MODE, M, OUT>(a, p, op, (wy * M + i) * 16, wx * M * 16, acc[i]);
  }
};

// ---------------------------------------------------------------------------
// Rows of whole 16-byte chunks go straight to LDS.  TY x TX tiles, WY x WX waves,
// steps of 128 bytes of z (whole lines; two matrix instructions deep), NS of
// them in LDS.  A wave holds the fragments of one half step while it reads the
// next half's, and the loads of step s + NS go out between the matrix
// instructions of the half in which step s has been read by all: one barrier
// per step, and no wave stands waiting to issue loads (in one burst they fill
// the CU's queue, and the wave with them).
// ---------------------------------------------------------------------------
template <int MODE, int TY_, int TX_, int WY, int WX, int NS, typename OUT>
struct Direct {
  static constexpr int TY = TY_, TX = TX_, KS = 2, NW = WY * WX, THREADS = 64 * NW;
  static constexpr int MY = TY / WY / 16, MX = TX / WX / 16;
  static constexpr int IY = TY * KS / 16 / NW, IX = TX * KS / 16 / NW, NI = IY + IX;   // loads of 1 KB per wave and step
  static constexpr int STEP = 64 * KS, STAGE = (TY + TX) * STEP;
  // FP4: E8M0 codes of 512 z, 16 bytes per row, two of such in turn
  static constexpr int SCALES = MODE == FOUR ? (TY + TX) * 16 : 0, IS = SCALES / 256 / NW;
  static constexpr int LDS = STAGE * NS + 2 * SCALES, PER_SIMD = 2;   // waves, by LDS and registers
  static constexpr int ZSTEP = (MODE == FOUR ? 128 : 32) * KS;
  static_assert(TY * KS / 16 % NW == 0 && TX * KS / 16 % NW == 0 && SCALES / 256 % NW == 0, "whole loads per wave");
  static_assert(MODE != FOUR || NS == 2, "the number of loads of a step varies");

  static __device__ __forceinline__ void dma16_base(uint32_t off, const uint8_t* base, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(lds) : "memory", "m0");
  }

  static __device__ __forceinline__ void run(const TileArgs& a, int64_t b, uint32_t lds) {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    Place p;
    if (!find_tile<MODE, TY, TX>(a, b, p)) return;
    const Operands<MODE> op(a, p);
    constexpr bool YT = Operands<MODE>::YT, XT = Operands<MODE>::XT;
    const int steps = pieces_of(op.zn, ZSTEP);
    const int full = op.zn / ZSTEP;   // steps without an end of z in them
    v4f acc[MY][MX];
#pragma unroll
    for (int i = 0; i < MY; ++i)
#pragma unroll
      for (int j = 0; j < MX; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

    // the lane's chunks of a step: bytes from the operand's place at that step.
    // Rows and columns past the extent: any others, never stored.
    uint32_t off[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool isy = i < IY;
      const int j = wave + NW * (isy ? i : i - IY);
      int row, chunk;
      if (isy) chunk_of<TY, YT, KS>(j, lane, row, chunk);
      else chunk_of<TX, XT, KS>(j, lane, row, chunk);
      const int extent = isy ? p.ny : p.nx, pitch = isy ? op.ybytes : op.xbytes;
      off[i] = (isy ? YT : XT) ? (uint32_t)row * pitch + min(chunk * 16, extent * 2 - 16)
                               : (uint32_t)min(row, extent - 1) * pitch + chunk * 16;
    }
    const uint8_t *yp = op.Y, *xp = op.X;   // at the next step to load
    const size_t ystep = YT ? (size_t)ZSTEP * op.ybytes : STEP, xstep = XT ? (size_t)ZSTEP * op.xbytes : STEP;
    auto place = [&](int i, uint32_t stage) {
      return stage + (i < IY ? (wave + NW * i) * 1024 : TY * STEP + (wave + NW * (i - IY)) * 1024);
    };
    auto load = [&](int i, int s, uint32_t stage, auto whole) {
      const uint8_t* base = i < IY ? yp : xp;
      if (decltype(whole)::value || s < full) {
        dma16_base(off[i], base, place(i, stage));
      } else {
        int row, chunk;
        const int j = wave + NW * (i < IY ? i : i - IY);
        if (i < IY) chunk_of<TY, YT, KS>(j, lane, row, chunk);
        else chunk_of<TX, XT, KS>(j, lane, row, chunk);
        const int z = (i < IY ? YT : XT) ? row : chunk * (MODE == FOUR ? 32 : 8);
        dma16(inside(s, ZSTEP, z, op.zn) ? base + off[i] : reinterpret_cast<const uint8_t*>(&zero_chunk), place(i, stage));
      }
    };
    // Every second tile takes the whole steps of a pair the other way round, so that
    // neighbours in step ask for different lines (2% on every product).
    auto z_of = [&](int s) { return (s | 1) < full ? s ^ p.odd : s; };
    auto advance = [&](int s) {
      const int z = z_of(s);
      yp = op.Y + (size_t)z * ystep;
      xp = op.X + (size_t)z * xstep;
    };
    advance(0);
    // FP4: the codes of steps s and s + 1, 4 lanes per row
    const uint8_t* xrow = a.X + ((size_t)p.e * a.N + p.x0) * op.xbytes;
    auto load_scales = [&](int s) {
      // of 128 z, from the slice's first on
      const int g = a.K / 32, word = 2 * s + (lane & 3), word0 = (int)(op.X - xrow) / 64;
#pragma unroll
      for (int i = 0; i < IS; ++i) {
        const int j = wave * IS + i, row = j * 16 + (lane >> 2);   // TY % 16 == 0: a load is of one operand
        const bool isy = j * 16 < TY;
        const uint8_t* q = isy ? a.SY + (size_t)(p.r0 + p.y0 + min(row, p.ny - 1)) * g
                               : a.SX + ((size_t)p.e * a.N + p.x0 + min(row - TY, p.nx - 1)) * g;
        vm_dma4(word * 128 < op.zn ? q + (word0 + word) * 4 : reinterpret_cast<const uint8_t*>(&zero_chunk),
                lds + STAGE * NS + ((s >> 1) & 1) * SCALES + j * 256);
      }
    };

    const int wy = wave / WX, wx = wave % WX;
    const int nb = ((p.ny + 15) / 16 - wy + WY - 1) / WY;   // the wave's row blocks: wy, wy + WY, ...
    v4i fy[4], fx[2][MX];
    uint32_t ey[MY], ex[MX];
    // addresses at stage 0: by half where z is contiguous
    const uint32_t y0 = lds + wy * 16 * STEP, x0 = lds + TY * STEP + wx * MX * 16 * STEP;
    const uint32_t ya[2] = {YT ? cols_base<TY>(lane) : rows_base<KS>(y0, 0, lane), YT ? 0 : rows_base<KS>(y0, 1, lane)};
    const uint32_t xa[2] = {XT ? cols_base<TX>(lane) : rows_base<KS>(x0, 0, lane), XT ? 0 : rows_base<KS>(x0, 1, lane)};
    auto read_y = [&](int h, int i, uint32_t stage) {
      fy[i & 3] = YT ? frag_cols<TY>(ya[0], lds + stage, i * WY + wy, h) : frag_rows<KS>(ya[h] + stage, i * WY);
    };
    auto read_x = [&](int h, int j, uint32_t stage) {
      fx[h][j] = XT ? frag_cols<TX>(xa[0], lds + stage + TY * STEP, wx * MX + j, h) : frag_rows<KS>(xa[h] + stage, j);
    };
    // The codes of the lane's blocks for the next 512 z, byte t of the t-th 128
    auto scales = [&](int s) {
      const uint32_t at = lds + STAGE * NS + ((s >> 1) & 1) * SCALES + (lane & 15) * 16;
      const uint32_t q = lane >> 4, sel = q | ((4 + q) << 8);
      auto word = [&](uint32_t row) {
        const v4i w = *(lds_v4i*)(uintptr_t)(at + row * 16);
        const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], sel), hi = __builtin_amdgcn_perm(w[3], w[2], sel);
        return __builtin_amdgcn_perm(hi, lo, z_of(s) == s ? 0x05040100u : 0x01000504u);
      };
#pragma unroll
      for (int i = 0; i < MY; ++i) ey[i] = word((i * WY + wy) * 16);
#pragma unroll
      for (int j = 0; j < MX; ++j) ex[j] = word(TY + (wx * MX + j) * 16);
    };
    auto multiply = [&](int h, int i) {   // row block i with half h
#pragma unroll
      for (int j = 0; j < MX; ++j) {
        if constexpr (MODE == FOUR) {
          const v8i x8 = {fx[h][j][0], fx[h][j][1], fx[h][j][2], fx[h][j][3], 0, 0, 0, 0};
          const v8i y8 = {fy[i & 3][0], fy[i & 3][1], fy[i & 3][2], fy[i & 3][3], 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x8, y8, acc[i][j], 4, 4, 0, (int)ex[j], 0, (int)ey[i]);
        } else {
          acc[i][j] = mfma_bf16(fx[h][j], fy[i & 3], acc[i][j]);
        }
      }
    };
    auto next_scales = [&]() {
      if constexpr (MODE == FOUR) {
#pragma unroll
        for (int i = 0; i < MY; ++i) ey[i] >>= 8;
#pragma unroll
        for (int j = 0; j < MX; ++j) ex[j] >>= 8;
      }
    };

    // Step s: groups g = 0 .. 2 MY - 1 of MX matrix instructions, one row block of
    // one half each.  Reads run AHEAD groups before their use; the loads of step
    // s + NS - 1 go out with the first groups (their place was read in step s -
    // 1); before the last AHEAD groups all waves have read step s and step s + 1
    // has landed.  WHOLE: the steps up to s + NS - 1 have all of their z; ALL: the
    // wave has all of its row blocks.
    constexpr int GROUPS = KS * MY, AHEAD = 2, EACH = std::max(2, (NI + GROUPS - AHEAD - 1) / (GROUPS - AHEAD));
    static_assert(MY >= 4, "four row blocks are held at a time");
    uint32_t stage = 0, spare = (NS - 1) * STAGE;
    auto step = [&](int s, auto whole_, auto all_) {
      constexpr bool WHOLE = decltype(whole_)::value, ALL = decltype(all_)::value;
      const bool two = WHOLE || inside(s, ZSTEP, ZSTEP / 2, op.zn);   // the second half has z
      const bool more = WHOLE || s + NS - 1 < steps, last = !WHOLE && s + 1 >= steps;
      const uint32_t after = stage == (NS - 1) * STAGE ? 0 : stage + STAGE;
      if (MODE == FOUR && !(s & 1)) scales(s);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const int h = g / MY, i = g % MY;
        if (g == GROUPS - AHEAD) {
          if (!last) {
            if (WHOLE || s + NS - 1 < steps) wait_and_meet<(NS - 2) * NI>();
            else wait_and_meet<0>();
#pragma unroll
            for (int j = 0; j < MX; ++j) read_x(0, j, after);
          }
        }
        if (g + AHEAD < GROUPS) {
          if (g + AHEAD < MY || two) read_y((g + AHEAD) / MY, (g + AHEAD) % MY, stage);
        } else if (!last) {
          read_y(0, g + AHEAD - GROUPS, after);
        }
        if (g < MY && two) {
#pragma unroll
          for (int j = 0; j < MX; ++j)
            if (j * (MY - 1) / MX == g) read_x(1, j, stage);   // spread over the first half
        }
        __builtin_amdgcn_sched_barrier(0);
        if ((ALL || i < nb) && (h == 0 || two)) multiply(h, i);
        __builtin_amdgcn_sched_barrier(0);
        if (more && g * EACH < NI) {
#pragma unroll
          for (int l = g * EACH; l < (g + 1) * EACH && l < NI; ++l) load(l, s + NS - 1, lds + spare, whole_);
          if (MODE == FOUR && (g + 1) * EACH >= NI && (s & 1)) load_scales(s + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (g == MY - 1 || g == GROUPS - 1) next_scales();
      }
      if (more) advance(s + NS);
      stage = after;
      spare = spare == (NS - 1) * STAGE ? 0 : spare + STAGE;
    };

#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      if (s < steps) {
#pragma unroll
        for (int i = 0; i < NI; ++i) load(i, s, lds + s * STAGE, std::false_type());
        advance(s + 1);
      }
    }
    if (MODE == FOUR) load_scales(0);
    if (MODE != FOUR && steps >= NS - 1) wait_and_meet<(NS - 2) * NI>();
    else wait_and_meet<0>();
    if (steps > 0) {
#pragma unroll
      for (int j = 0; j < MX; ++j) read_x(0, j, 0);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) read_y(0, i, 0);
    }
    int s = 0;
    if (nb == MY)
      for (; s + NS - 1 < full; ++s) step(s, std::true_type(), std::true_type());
    else
      for (; s + NS - 1 < full; ++s) step(s, std::true_type(), std::false_type());
    for (; s < steps; ++s) step(s, std::false_type(), std::false_type());

    if (MODE == WEIGHTS && a.accumulate && steps == 0) return;
#pragma unroll
    for (int i = 0; i < MY; ++i)
      put_block<MODE, MX, OUT>(a, p, op, (i * WY + wy) * 16, wx * MX * 16, acc[i]);
  }
};

template <typename T>
__global__ void __launch_bounds__(T::THREADS, T::PER_SIMD)
tile_kernel(TileArgs a, int64_t b0) {
  extern __shared__ __align__(1024) uint8_t smem[];
  T::run(a, b0 + blockIdx.x, lds_u32(smem));
}

// Workgroups of a product: tiles are known for the weights, otherwise at most
// (each expert's last may be part of one); they come in eights, one per XCD.
template <int MODE>
int64_t workgroups(const TileArgs& a, int TY, int TX) {
  const int64_t width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N, nt = (width + TX - 1) / TX;
  const int64_t eights = MODE == WEIGHTS ? a.E * (((a.N + TY - 1) / TY * nt + 7) / 8)
                                         : ((a.R + (int64_t)std::min(a.E, a.R) * (TY - 1)) / TY * nt + 7) / 8;
  return eights * 8;
}

template <int MODE, typename T>
hipError_t launch(const TileArgs& a, hipStream_t stream) {
  if (T::LDS > 64 * 1024) {
    // more than a launch has without asking; once per device
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (!(allowed.load(std::memory_order_acquire) & bit)) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(&tile_kernel<T>), hipFuncAttributeMaxDynamicSharedMemorySize,
                              T::LDS);
      if (e != hipSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_release);
    }
  }
  return in_launches(workgroups<MODE>(a, T::TY, T::TX), T::THREADS, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(tile_kernel<T>, dim3((unsigned)n, a.slices), dim3(T::THREADS), T::LDS, stream, a, b);
  });
}

// The slices' sums to the output, in the slices' order: flat, from the first row
// on to the last that the offsets give.
template <int MODE, typename OUT>
__global__ void __launch_bounds__(256)
join_kernel(TileArgs a, const float* __restrict__ parts) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
    const int o0 = a.offsets[i], o1 = a.offsets[i + 1];
    if (o1 < o0 || (i == 0 && o0 != 0) || (i == a.E - 1 && o1 > a.R)) bad = 1;
  }
  __syncthreads();
  if (bad) return;
  const size_t width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N;
  const size_t all = (MODE == WEIGHTS ? (size_t)a.E * a.N : (size_t)a.R) * width;
  const size_t n = MODE == WEIGHTS ? all : (size_t)a.offsets[a.E] * width;
  OUT* out = static_cast<OUT*>(a.out);
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
    float v = 0.f;
    for (int s0 = 0; s0 < a.slices; s0 += 16) {   // 16 loads on their way
      float part[16];
#pragma unroll
      for (int s = 0; s < 16; ++s) part[s] = s0 + s < a.slices ? parts[(s0 + s) * all + i] : 0.f;
#pragma unroll
      for (int s = 0; s < 16; ++s) v += part[s];
    }
    if (MODE == WEIGHTS && a.accumulate)
      v += sizeof(OUT) == 4 ? (float)out[i] : __uint_as_float((uint32_t)(uint16_t)out[i] << 16);
    if constexpr (sizeof(OUT) == 4) out[i] = v;
    else out[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename OUT>
bool wide_out(const TileArgs& a, int width) { return width % (16 / sizeof(OUT)) == 0 && aligned_to(a.out, 16); }

// Where a product has fewer tiles than the chip has CUs and a long sum, the sum is
// cut into slices (parts of fp32 in the workspace, added in order): 3 rows, 128 x
// 5969, 112 us in one piece and 18 in 23; the row gradient of 36 rows, 4848 x 102,
// 246 and 19.
template <int MODE, typename OUT, typename F>
hipError_t launch_sliced(TileArgs a, void* work, hipStream_t stream, F launch_tiles) {
  const int width = MODE == ROWS || MODE == WEIGHTS ? a.K : a.N;
  a.slices = work ? product_slices(MODE, a.R, a.E, a.N, a.K) : 1;
  if (a.slices == 1) {
    a.wide = wide_out<OUT>(a, width);
    return launch_tiles(a, OUT());
  }
  TileArgs part = a;
  part.out = work;
  part.accumulate = 0;
  part.wide = wide_out<float>(part, width);
  const hipError_t e = launch_tiles(part, float());
  if (e != hipSuccess) return e;
  const int64_t n = (MODE == WEIGHTS ? (int64_t)a.E * a.N : (int64_t)a.R) * width;
  const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 2048);
  hipLaunchKernelGGL((join_kernel<MODE, OUT>), dim3(grid), dim3(256), 0, stream, a, static_cast<const float*>(work));
  return hipGetLastError();
}

// Steps of 64 z where the forward product's operands lie along z, and for few rows,
// which read most of what they load once; steps of 32, with three workgroups on a CU
// in place of two, for the others.  us, 64 | 32: forward, 9216 rows, 32 experts 4096 x
// 2047 387 | 422, 88 rows, 29 experts 2554 x 3266 117 | 130; row gradient, 88 rows, 29
// experts 2553 x 1266 75 | 98, 97704 rows, 9 experts 838 x 401 219 | 205; weights'
// gradient, 65536 rows, 8 experts 1447 x 1025 501 | 430.
template <int MODE, typename OUT>
hipError_t launch_odd(const TileArgs& a, hipStream_t stream) {
  if constexpr (MODE != WEIGHTS)
    if (MODE == FWD || a.R / a.E <= FEW_ROWS) return launch<MODE, General<MODE, 2, OUT>>(a, stream);
  if constexpr (MODE != FWD) return launch<MODE, General<MODE, 1, OUT>>(a, stream);
}

// Tiles by the mean number of rows of an expert (all that the host knows).
// 4096 x 6144, 32 experts, unevenly filled, us a call, forward | row gradient:
//   rows        16          64          128         288          512          1024
//   64 x 128    273 | 279   368 | 365   479 | 471   824 | 787    1344 | 1285  2545 | 2437
//   128 x 256   273 | 263   342 | 322   416 | 384   601 | 586     925 | 901   1688 | 1666
//   256 x 256   340 | 319   367 | 342   496 | 439   667 | 646     975 | 888   1639 | 1581
// Where tiles are few, the small ones fill the chip (forward, 12 experts of 43
// rows, 6144 x 3584: 113 against 129 us); the row gradient reads whole lines of
// the weights only with 256 columns (127 against 103).  The weights' gradient has
// its largest tiles at any number of rows (16: 671 against 750 us with 128 x 256,
// 288: 1133 / 1253, 1024: 2070 / 2282).
// A tile also needs enough of its kind: if there are half as many as CUs or fewer, the
// next smaller ones are done in one round as well, in less time (8 experts, 8192 rows,
// 512 x 4096: forward 80 us with the largest, 47; 4 by 4 bits 34, 20; 7384 rows, 256 x
// 2864, forward 49, 24; but 24000 rows, 512 x 2048: 48, 58 with 1.5 rounds).  The width
// is not looked at: 57085 rows, 60 experts 128 x 640, 4 by 4 bits take the largest, half
// empty, 23 us.
enum { SMALL, MIDDLE, LARGE, ODD };
struct TileSize { int y, x; };
constexpr TileSize size_of(int mode, int tile) {
  return tile == SMALL ? TileSize{64, 128} : tile == LARGE ? TileSize{256, 256}
         : tile == MIDDLE && mode != FOUR ? TileSize{128, 256} : TileSize{128, 128};
}
template <int MODE, int TILE, typename OUT>
using DirectTile = Direct<MODE, size_of(MODE, TILE).y, size_of(MODE, TILE).x, TILE == SMALL ? 1 : 2,
                          MODE == FOUR && TILE == MIDDLE ? 2 : 4, MODE == FOUR || TILE == LARGE ? 2 : 3, OUT>;
// Tiles whose sums product_slices() may cut: the others come in numbers that fill
// the chip, and their kernels for parts in fp32 do not exist.
constexpr bool in_slices(int mode, int tile) {
  return tile == ODD || mode == WEIGHTS || tile == (mode == ROWS ? MIDDLE : SMALL) || (mode == FOUR && tile == MIDDLE);
}
template <int MODE, int TILE, typename OUT>
hipError_t launch_tile(const TileArgs& a, hipStream_t stream) {
  if constexpr (sizeof(OUT) == 4 && !in_slices(MODE, TILE)) return hipErrorInvalidValue;
  else return launch<MODE, DirectTile<MODE, TILE, OUT>>(a, stream);
}
template <int MODE>
int tile_of(const TileArgs& a) {
  const int rows = a.R / a.E;
  if (MODE == FOUR) {
    // as above; 16 rows: 84, 88 and 108 us with these three, 64: 134, 125 and 125,
    // 128: 186, 159 and 170, 288: 311, 243 and 239, 1024: 882, 671 and 576
    if (rows <= 32) return SMALL;
    return rows <= 200 || workgroups<MODE>(a, 256, 256) <= CUS / 2 ? MIDDLE : LARGE;
  }
  if (MODE == WEIGHTS) return LARGE;
  if (MODE == FWD && (rows <= FEW_ROWS || workgroups<MODE>(a, 128, 256) <= CUS / 2)) return SMALL;
  return rows <= MANY_ROWS || workgroups<MODE>(a, 256, 256) <= CUS / 2 ? MIDDLE : LARGE;
}

int tile_for(int mode, const TileArgs& a) {
  return mode == FWD ? tile_of<FWD>(a) : mode == ROWS ? tile_of<ROWS>(a) : mode == WEIGHTS ? tile_of<WEIGHTS>(a)
                                                                                           : tile_of<FOUR>(a);
}

// Whole chunks: along K of the forward product's rows, along both of the others.
// A tile's offsets within an operand are 32 bits: 256 rows, or 64 of z, of 8 MB
// at most.
bool odd_sizes(int mode, int N, int K) {
  return mode != FOUR && (K % 8 || (mode != FWD && N % 8) || N > (1 << 22));
}

template <int MODE, typename OUT>
hipError_t launch_bf16(const TileArgs& a, hipStream_t stream) {
  if (odd_sizes(MODE, a.N, a.K) || !aligned_to(a.Y, 16) || !aligned_to(a.X, 16))
    return launch_odd<MODE, OUT>(a, stream);
  const int tile = tile_of<MODE>(a);
  if constexpr (MODE == FWD)
    if (tile == SMALL) return launch_tile<MODE, SMALL, OUT>(a, stream);
  if constexpr (MODE != WEIGHTS)
    if (tile == MIDDLE) return launch_tile<MODE, MIDDLE, OUT>(a, stream);
  return launch_tile<MODE, LARGE, OUT>(a, stream);
}

template <typename OUT>
hipError_t launch_four(const TileArgs& a, hipStream_t stream) {
  const int tile = tile_of<FOUR>(a);
  if (tile == SMALL) return launch_tile<FOUR, SMALL, OUT>(a, stream);
  if (tile == MIDDLE) return launch_tile<FOUR, MIDDLE, OUT>(a, stream);
  return launch_tile<FOUR, LARGE, OUT>(a, stream);
}

}  // namespace

// Slices of a sum: as many as bring the workgroups to the number that the chip holds
// at a time, none shorter than `least`, and none at all below `from`, where the join's
// launch costs what they give.  One piece | slices, us: forward, 8 experts 1024 x 512
// 6.7 | 9.0 in 2, x 1024 9.1 | 9.6 in 3, x 2048 14.2 | 11.6 in 3; row gradient, 2
// experts 1024 x 512 14.8 | 12.6 in 4; 4 by 4 bits, 8 experts 1024 x 2048 8.7 | 10.7
// in 2, x 4096 13.2 | 12.2 in 3, x 8192 29.3 | 17.7 in 3.  Odd sizes: 8 experts 1024
// x 1023 25.5 | 15.2 in 3.
int product_slices(int mode, int R, int E, int N, int K) {
  if (R < 1) return 1;
  TileArgs a{};
  a.R = R;
  a.E = E;
  a.N = N;
  a.K = K;
  const int rows = R / E;
  const bool odd = mode != FOUR && (K % 8 || (mode != FWD && N % 8));   // 128 x 128, two workgroups on a CU
  if (!odd && !in_slices(mode, tile_for(mode, a))) return 1;
  int64_t tiles, z, out, most = 1 << 22;   // values of all parts: 16 MB take no longer than a launch
  int least = 256, from = 1024;
  if (mode == FWD) {
    tiles = odd ? workgroups<FWD>(a, 128, 128) : workgroups<FWD>(a, 64, 128);
    z = K;
    out = (int64_t)R * N;
  } else if (mode == ROWS) {
    tiles = odd ? workgroups<ROWS>(a, 128, 128) : workgroups<ROWS>(a, 128, 256);
    z = N;
    out = (int64_t)R * K;
  } else if (mode == WEIGHTS) {
    // one expert may have most of the rows: slices as if it were four times the
    // mean, up to four times the workgroups, and parts of up to 1 KB for each row (46000
    // rows unevenly to 26 experts, 1446 x 62: 1465 us in one piece, 133 in 4)
    const int64_t edge = odd ? 128 : 256;
    tiles = (E * ((N + edge - 1) / edge) * ((K + edge - 1) / edge) + 3) / 4;
    z = std::min<int64_t>(R, (int64_t)rows * 4);
    most = std::max<int64_t>(most, (int64_t)R << 8);
    from = 2048;
    out = (int64_t)E * N * K;
  } else {
    tiles = tile_of<FOUR>(a) == SMALL ? workgroups<FOUR>(a, 64, 128) : workgroups<FOUR>(a, 128, 128);
    z = K;
    out = (int64_t)R * N;
    least = 1024;
    from = 4096;
  }
  if (odd) from /= 2;
  if (z < from) return 1;
  const int64_t at_a_time = odd ? 2 * CUS : CUS;
  const int64_t s = std::min({(int64_t)64, z / least, at_a_time / tiles, most / std::max<int64_t>(1, out)});
  return (int)std::max<int64_t>(1, s);
}

int product_tile(int mode, int R, int E, int N, int K) {
  TileArgs a{};
  a.R = R;
  a.E = E;
  a.N = N;
  a.K = K;
  const int tile = odd_sizes(mode, N, K) ? ODD : tile_for(mode, a);
  return size_of(mode, tile).y << 16 | size_of(mode, tile).x;
}

size_t product_workspace(int mode, int R, int E, int N, int K) {
  const int s = product_slices(mode, R, E, N, K);
  const size_t out = mode == FWD || mode == FOUR ? (size_t)R * N : mode == ROWS ? (size_t)R * K : (size_t)E * N * K;
  return s == 1 ? 0 : s * out * sizeof(float);
}

hipError_t launch_grouped_bf16(const TileArgs& a, void* work, hipStream_t stream) {
  return launch_sliced<FWD, uint16_t>(a, work, stream, [&](const TileArgs& t, auto out) {
    return launch_bf16<FWD, decltype(out)>(t, stream);
  });
}
hipError_t launch_grouped_dgrad(const TileArgs& a, void* work, hipStream_t stream) {
  return launch_sliced<ROWS, uint16_t>(a, work, stream, [&](const TileArgs& t, auto out) {
    return launch_bf16<ROWS, decltype(out)>(t, stream);
  });
}
hipError_t launch_grouped_wgrad(const TileArgs& a, bool f32, void* work, hipStream_t stream) {
  const auto tiles = [&](const TileArgs& t, auto out) { return launch_bf16<WEIGHTS, decltype(out)>(t, stream); };
  return f32 ? launch_sliced<WEIGHTS, float>(a, work, stream, tiles)
             : launch_sliced<WEIGHTS, uint16_t>(a, work, stream, tiles);
}
hipError_t launch_grouped_a4(const TileArgs& a, void* work, hipStream_t stream) {
  return launch_sliced<FOUR, uint16_t>(a, work, stream, [&](const TileArgs& t, auto out) {
    return launch_four<decltype(out)>(t, stream);
  });
}

}  // namespace w4a8
