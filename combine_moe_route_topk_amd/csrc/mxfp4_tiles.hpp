// How many tiles the MXFP4 tile kernel makes: the rule of the kernel, which
// counts the row tiles that exist, and of its launch, which knows a bound on
// them alone.  Plain host code (constexpr functions are device code, too).
#pragma once

#include <stdint.h>

namespace moe {
namespace {
namespace big {

constexpr int kBM = 256;               // rows of a tile
constexpr int64_t kFewTiles = 128;     // half the CUs: up to as many tiles have half the columns

// Tiles of n columns: 256 wide, 128 with SwiGLU, or half of that.
constexpr int64_t col_tiles(int64_t n, bool glu, bool few) {
  return glu ? (few ? (n + 63) / 64 : (n + 127) / 128) : (few ? (n + 127) / 128 : (n + 255) / 256);
}

// any: the kernel's form that can halve the columns.
constexpr bool few_tiles(int64_t row_tiles, int64_t n, bool glu, bool any) {
  return any && row_tiles * col_tiles(n, glu, false) <= kFewTiles;
}

// Tiles that the kernel makes of `row_tiles` that exist.
constexpr int64_t tiles_of(int64_t row_tiles, int64_t n, bool glu, bool any) {
  return row_tiles * col_tiles(n, glu, few_tiles(row_tiles, n, glu, any));
}

// Workgroups that hold every tile whatever number of row tiles up to `most`
// exists.  The number of tiles is not monotone: just below kFewTiles it is twice
// that of wide tiles, so most row tiles can need fewer workgroups than some
// smaller number, which rows without an expert leave.
constexpr int64_t blocks_for(int64_t most, int64_t n, bool glu, bool any) {
  const int64_t wide = col_tiles(n, glu, false);
  const int64_t few = any ? (most < kFewTiles / wide ? most : kFewTiles / wide) : 0;
  const int64_t a = most * wide, b = few * col_tiles(n, glu, true);
  return a > b ? a : b;
}

}  // namespace big
}  // namespace
}  // namespace moe
