// Index arithmetic of the tiled products, by itself so that it also compiles
// without HIP.  Rows and sums go up to 2^31 - 1: what adds a tile or a step to
// them does so in unsigned 32 bits, which hold it.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define W4A8_HD __host__ __device__
#else
#define W4A8_HD
#endif

namespace w4a8 {

// Tiles (steps) of `size` that n rows (z) take; n >= 0.
W4A8_HD constexpr int pieces_of(int n, int size) {
  return (int)(((uint32_t)n + (uint32_t)(size - 1)) / (uint32_t)size);
}

// Rows of each tile where `rows` go to `tiles` tiles evenly, in whole blocks of
// 16; with tiles = pieces_of(rows, T) and T a multiple of 16, at most T, and the
// last tile has a row: (tiles - 1) * T < rows.
W4A8_HD constexpr int rows_per_tile(int rows, int tiles) {
  return (int)((((uint32_t)rows + (uint32_t)(tiles - 1)) / (uint32_t)tiles + 15u) & ~15u);
}

// Whether place `at` of step s is inside z (s < pieces_of(z, step), 0 <= at < step).
W4A8_HD constexpr bool inside(int s, int step, int at, int z) {
  return (uint32_t)s * (uint32_t)step + (uint32_t)at < (uint32_t)z;
}

// z of a slice, whole steps; slices * this > z, slices >= 2.  The last slice's
// start is in 32 bits: (slices - 1) * this is at most z - z / slices + (slices -
// 1) * step.
W4A8_HD constexpr int slice_of(int z, int slices, int step) { return (z / slices + step) / step * step; }

}  // namespace w4a8
