// Device types and helpers shared by the matrix product's kernels (product*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_internal.h"
#include "load_bounds.h"

namespace mxfp8 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// LDS: the 32-bit address of a generic pointer's object, and an object at such an address.
#define LDS_AT(T, at) ((__attribute__((address_space(3))) T*)(uintptr_t)(at))
#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T*)(p))

constexpr int kStep = 128;   // values of the sum per step
constexpr int kGroup = 4;    // steps whose scales are staged together (16 bytes per row)

struct Operand {
  const uint8_t* data;
  const uint8_t* scale;
  int64_t ld;
  int64_t outer;         // valid rows (ALONG_COLS) or columns (ALONG_ROWS) of the array
  int64_t s_outer;       // scale strides: per scale row, per scale block along the sum
  int64_t s_block;
  int across_shift;      // log2 of outer values per scale
  int block_shift;       // log2 of 32-value blocks per scale: 0 or 2
};

struct ProductArgs {
  Operand a, b;
  int64_t m, n, k;
  void* out;
  int64_t ldo;
  const float* add;
  int64_t ldadd;
  float* part;           // [splits][m][n] when the sum is split
  int64_t steps;         // steps per part
  int tiles_m, tiles_n;
  uint8_t* packed;       // large tiles: the operands' scales, [2][group][row][16]
};

// ---------------------------------------------------------------- scales
//
// Staged per group of 4 steps: for each outer row 4 dwords, dword j holding the scale bytes of
// 32-value block j of the group's steps 0..3.  Rows and blocks past the end take the last valid
// one's: such rows are not stored, and such blocks' codes are 0.

struct ScaleBytes {
  uint32_t w[4];  // byte e of the group's 16 blocks (block 32), or w[0] = 4 bytes (block 128)
};

__device__ inline ScaleBytes load_scales(const Operand& o, int64_t outer, int64_t k,
                                         int64_t group) {
  ScaleBytes s = {{0, 0, 0, 0}};
  outer = outer < o.outer ? outer : o.outer - 1;
  const uint8_t* p = o.scale + (outer >> o.across_shift) * o.s_outer;
  if (o.block_shift == 0) {
    const int last = (int)((k + 31) / 32) - 1, first = (int)group * 16;
    if (o.s_block == 1 && first + 15 <= last) {
      __builtin_memcpy(s.w, p + first, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        s.w[e / 4] |= (uint32_t)p[min(first + e, last) * o.s_block] << (8 * (e % 4));
    }
  } else {
    const int last = (int)((k + 127) / 128) - 1, first = (int)group * 4;
    if (o.s_block == 1 && first + 3 <= last) {
      __builtin_memcpy(s.w, p + first, 4);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s.w[0] |= (uint32_t)p[min(first + e, last) * o.s_block] << (8 * e);
    }
  }
  return s;
}

__device__ inline v4i arrange_scales(const ScaleBytes& s, int block_shift) {
  if (block_shift) return v4i{(int)s.w[0], (int)s.w[0], (int)s.w[0], (int)s.w[0]};
  v4i d;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) v |= ((s.w[t] >> (8 * j)) & 0xFF) << (8 * t);
    d[j] = (int)v;
  }
  return d;
}

// Which output tile a workgroup computes.  Successive workgroups go to the 8 XCDs in turn, so
// each XCD takes a contiguous part of the tiles, in bands of 4 tile rows: the 32 tiles its CUs
// work on at a time are 4 x 8 and share their operands in the XCD's L2.
__device__ inline void tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int tiles = tiles_m * tiles_n, xcd = id & 7, rank = id >> 3;
  const int each = tiles >> 3, extra = tiles & 7;
  const int t = xcd * each + (xcd < extra ? xcd : extra) + rank;
  const int band = t / (4 * tiles_n), rows = tiles_m - 4 * band < 4 ? tiles_m - 4 * band : 4;
  const int in = t - band * 4 * tiles_n;
  tm = 4 * band + in % rows;
  tn = in / rows;
}

__device__ inline v8b to_bf16(int lo, int hi, float scale) {
  const v2b a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const v2b b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const v2b c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const v2b d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return v8b{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ inline void barrier() { asm volatile("s_barrier" ::: "memory"); }

__device__ inline uint16_t bf16_bits(float x) {
  const __bf16 b = (__bf16)x;  // nearest even
  return __builtin_bit_cast(uint16_t, b);
}

// For m <= 16, both operands ALONG_COLS (product_few.hip).
hipError_t launch_few(const ProductArgs& g, bool f32, hipStream_t s);

// The main kernel (product_pack.hip), and its tile sizes (two files each); `ar`, `br`: the operands
// are ALONG_ROWS.
hipError_t launch_large_product(ProductArgs g, const ProductPlan& plan, bool ar, bool br, bool f32,
                                hipStream_t s);
hipError_t launch_256x256(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_256x256_fp32(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_256x192(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_256x192_fp32(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_128x128(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_128x128_fp32(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_64x128(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);
hipError_t launch_64x128_fp32(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s);

}  // namespace mxfp8
