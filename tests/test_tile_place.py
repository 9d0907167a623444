"""The tiled products' index arithmetic, compiled for the host: against the same
in 64 bits, up to the largest number of rows and the longest sum that a call may
have (2^31 - 1)."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_grouped_precision_amd", "csrc")

PROGRAM = r"""
#include "tile_place.h"
#include <cstdint>
#include <cstdio>
using namespace w4a8;
#define CHECK(what) do { if (!(what)) { std::printf("%s: n=%lld size=%lld\n", #what, (long long)n, (long long)size); return 1; } } while (0)

static int rows(int64_t n, int64_t size) {
  const int64_t tiles = (n + size - 1) / size;
  CHECK(pieces_of((int)n, (int)size) == tiles);
  if (tiles == 0) return 0;
  const int64_t per = ((n + tiles - 1) / tiles + 15) / 16 * 16;
  CHECK(rows_per_tile((int)n, (int)tiles) == per);
  CHECK(per <= size && (tiles - 1) * per < n && tiles * per >= n);   // every row in one tile, none empty
  return 0;
}
static int z(int64_t n, int64_t size) {
  const int64_t steps = (n + size - 1) / size;
  for (int64_t s = steps > 3 ? steps - 3 : 0; s < steps; ++s)
    for (int64_t at = 0; at < size; ++at) CHECK(inside((int)s, (int)size, (int)at, (int)n) == (s * size + at < n));
  for (int64_t slices = 2; slices <= 64; ++slices) {
    const int64_t each = (n / slices + size) / size * size;
    CHECK(slice_of((int)n, (int)slices, (int)size) == each && slices * each > n);
    CHECK((slices - 1) * each <= INT32_MAX);
  }
  return 0;
}
int main() {
  const int64_t last = INT32_MAX, ends[] = {0, 1, 48, 63, 64, 65, 1000, 4097, 1 << 20, last / 2, 2139500000, 2140000000, last};
  const int64_t sizes[] = {32, 64, 128, 256, 512};
  for (int64_t end : ends)
    for (int64_t n = end > 700 ? end - 700 : 0; n <= end; ++n)
      for (int64_t size : sizes) {
        if (size >= 64 && size <= 256 && rows(n, size)) return 1;
        if (z(n, size)) return 1;
      }
  for (int64_t i = 0; i < 300000; ++i) {
    const int64_t n = (i * 2654435761ll + 12345) % (last + 1);
    for (int64_t size : sizes)
      if (size >= 64 && size <= 256 && rows(n, size)) return 1;
  }
  std::puts("ok");
  return 0;
}
"""


def test_rows_and_sums_up_to_32_bits(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "place.cpp", tmp_path / "place"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-ftrapv", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout == "ok\n", res.stdout
