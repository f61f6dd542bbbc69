// Which bytes the matrix product's main kernel loads (product_large.h): where each 16-byte slot of
// a half step's LDS buffer comes from, and how far the half's buffer resource reaches.  Plain C++
// without HIP, so that a host program can replay every load.
#pragma once

#include <stdint.h>

namespace mxfp8 {

constexpr int kHalf = 64;  // values of the sum per phase

// Swizzle of a tile stored along the rows of its array; see each kernel's LDS layout.
template <int T>
constexpr int rows_swizzle(int k) {
  constexpr int chunks = T / 16;
  if constexpr (chunks == 12) return 2 * ((k >> 2) & 1);  // rows 48 banks apart: 4 of them cover all
  constexpr int sh = chunks >= 16 ? 0 : chunks == 8 ? 1 : chunks == 4 ? 2 : 3;
  return (2 * ((k & 7) >> sh)) & (chunks - 1);
}

// The array row, from the half's base on, and the byte in it that slot `slot` is loaded from.
struct Place {
  int row, at;
};
template <int T, bool kRows>
constexpr Place place_of(int slot) {
  if constexpr (kRows) {
    constexpr int chunks = T / 16;
    const int k = slot / chunks;
    return {k, 16 * ((slot % chunks) ^ rows_swizzle<T>(k))};
  } else {
    const int r = slot / 4;
    return {r, 16 * ((slot % 4) ^ ((r >> 2) & 3))};
  }
}

// ALONG_COLS: bytes from the half's base that its loads may touch, with `rows` rows of the array
// from the tile's first on (at most T count).  The last row ends after min(64, ld) bytes: a row
// past it starts ld bytes on, so none of it is inside, however short the rows are.
template <int T>
constexpr uint32_t cols_extent(int64_t rows, int64_t ld) {
  return (uint32_t)(((rows < T ? rows : T) - 1) * ld + (ld < kHalf ? ld : kHalf));
}

// Which of a row's bytes belong to the sum is checked for each lane: those that start `left` or more
// values on take an offset past every extent, and so read 0.
constexpr uint32_t cols_offset(uint32_t offset, int at, int left) { return at < left ? offset : 0xFFFFFFF0u; }

// ALONG_ROWS: the extent, with `left` values of the sum from the half's start on and `width` columns
// of the array from the tile's first on.
constexpr uint32_t rows_extent(int left, int ld, int64_t width) {
  return left > 0 ? (uint32_t)((left < kHalf ? left : kHalf) - 1) * (uint32_t)ld + (uint32_t)width : 0u;
}

}  // namespace mxfp8
