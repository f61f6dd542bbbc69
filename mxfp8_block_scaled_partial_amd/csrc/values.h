// Device helpers shared by the activation and layer-norm kernels: chunks of 8 successive
// values of a row in FP32 registers, whatever their type and alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxfp8 {

struct Chunk {
  float v[8];
};

__device__ inline uint32_t bf16_round(float x) {  // nearest even; NaN stays NaN
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

// 16 and 8 bytes at any alignment.  Streaming accesses carry the non-temporal hint: outputs are
// written once and not read here; the activation's inputs are read once and dropped.  With inputs
// that change from call to call, without and with the stores' hint: layer norm of 16384 x 6144 BF16
// 86.6 and 84.3 us forward, 145.4 and 142.4 backward, SwiGLU of 8192 x 14336 BF16 210 and 206 forward,
// 238 and 240 backward; the loads' hint: SwiGLU backward 244 and 240.  (With the same inputs every
// call layer norm forward takes 89 and 69 us: the stores leave its inputs in the cache.)  Layer
// norm's loads do without: its inputs are read again by the backward pass.
typedef uint32_t Bytes16 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t Bytes8 __attribute__((ext_vector_type(2), aligned(1)));

template <bool kStream>
__device__ inline Bytes16 load16(const void* p) {
  const auto* q = static_cast<const Bytes16*>(p);
  if constexpr (kStream) return __builtin_nontemporal_load(q);
  return *q;
}
template <bool kStream>
__device__ inline void store16(void* p, const uint32_t* w) {
  const Bytes16 v = {w[0], w[1], w[2], w[3]};
  auto* q = static_cast<Bytes16*>(p);
  if constexpr (kStream)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// 8 values as they lie in memory.
template <bool kBF16>
struct Raw {
  uint32_t w[kBF16 ? 4 : 8];
};

// 8 values from base + index on, of which the first `valid` exist; the rest become 0.  A whole
// chunk is one or two 16-byte loads (global loads need no alignment).
template <bool kBF16, bool kStream = false>
__device__ inline Raw<kBF16> load_raw(const void* base, int64_t index, int64_t valid) {
  Raw<kBF16> r;
  const auto* p = static_cast<const uint8_t*>(base) + index * (kBF16 ? 2 : 4);
  if (valid >= 8) {
#pragma unroll
    for (int i = 0; i < (kBF16 ? 1 : 2); ++i) {
      const Bytes16 v = load16<kStream>(p + 16 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[4 * i + e] = v[e];
    }
  } else if constexpr (kBF16) {
    const auto* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.w[i] = (2 * i < valid ? q[2 * i] : 0u) | (2 * i + 1 < valid ? (uint32_t)q[2 * i + 1] << 16 : 0u);
  } else {
    const auto* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = i < valid ? q[i] : 0u;
  }
  return r;
}

template <bool kBF16>
__device__ inline Chunk values_of(const Raw<kBF16>& r) {
  Chunk c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kBF16)
      c.v[i] = __uint_as_float(i % 2 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
    else
      c.v[i] = __uint_as_float(r.w[i]);
  }
  return c;
}

template <bool kBF16>
__device__ inline Chunk load8(const void* base, int64_t index, int64_t valid) {
  return values_of<kBF16>(load_raw<kBF16>(base, index, valid));
}

template <bool kBF16, bool kStream = true>
__device__ inline void store8(void* base, int64_t index, int64_t valid, const Chunk& c) {
  if constexpr (kBF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + index;
    if (valid >= 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = bf16_round(c.v[2 * i]) | bf16_round(c.v[2 * i + 1]) << 16;
      store16<kStream>(p, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) p[i] = (uint16_t)bf16_round(c.v[i]);
    }
  } else {
    float* p = static_cast<float*>(base) + index;
    if (valid >= 8) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(c.v[i]);
      store16<kStream>(p, w);
      store16<kStream>(p + 4, w + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid) p[i] = c.v[i];
    }
  }
}

// 8 bytes (E4M3 codes) at p + index, the first `valid` of which belong to the row.
__device__ inline void store8_bytes(uint8_t* p, int64_t index, int64_t valid, uint2 w) {
  if (valid >= 8) {
    __builtin_nontemporal_store(Bytes8{w.x, w.y}, reinterpret_cast<Bytes8*>(p + index));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[index + i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i % 4)));
  }
}

__device__ inline uint2 load8_bytes(const uint8_t* p, int64_t index, int64_t valid) {
  uint2 w = {0, 0};
  if (valid >= 8) {
    const Bytes8 v = __builtin_nontemporal_load(reinterpret_cast<const Bytes8*>(p + index));
    w = {v[0], v[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) {
        if (i < 4)
          w.x |= (uint32_t)p[index + i] << (8 * i);
        else
          w.y |= (uint32_t)p[index + i] << (8 * (i - 4));
      }
  }
  return w;
}

// Bits of |x| for an amax over finite values: 0 for an infinity or NaN.
__device__ inline uint32_t finite_bits(float x) {
  const uint32_t a = __float_as_uint(x) & 0x7FFFFFFFu;
  return a < 0x7F800000u ? a : 0u;
}

// E8M0 byte of an amax (its FP32 bits, finite): max(0, exponent field - 8).
__device__ inline uint32_t scale_of(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e > 8 ? e - 8 : 0;
}

// 2^(127 - s) for a scale byte s <= 253, exactly.
__device__ inline float scale_up(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// A value ready for the E4M3 conversion: scaled, saturated to +-448; an infinity or NaN
// becomes a NaN, whose code the conversion makes 0xFF.
__device__ inline float to_e4m3_range(float x, float up) {
  const float y = __builtin_amdgcn_fmed3f(x * up, -448.f, 448.f);
  const bool finite = (__float_as_uint(x) & 0x7FFFFFFFu) < 0x7F800000u;
  return finite ? y : __uint_as_float(0x7FC00000u);
}

// ---- the same for blocks of ordinary values: every value finite, and a scale byte of 0 only
// where all are 0.  The conversion then applies the scale itself (v_cvt_scalef32_pk_fp8_f32
// divides by a power of two) and, with MODE.FP16_OVFL set, saturates to +-448: half an
// instruction per value where the general form takes five.

constexpr uint32_t kInfinity = 0x7F800000u;

// Sets MODE.FP16_OVFL (bit 23) for the wave: conversions to E4M3 saturate.
__device__ inline void saturate_conversions() { __builtin_amdgcn_s_setreg(1 | 23 << 6 | 0 << 11, 1); }

// Bits of |x|: an infinity or NaN compares as at least kInfinity.
__device__ inline uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Whether a block with this amax (bits, infinities and NaN included) needs the general form.
__device__ inline bool unusual(uint32_t amax) {
  return amax >= kInfinity || (amax != 0 && scale_of(amax) == 0);
}

// 2^(s - 127) of an ordinary block: s = 0 holds only zeros, for which any factor will do.
__device__ inline float scale_factor(uint32_t s) { return __uint_as_float((s ? s : 127u) << 23); }

typedef short v2s __attribute__((ext_vector_type(2)));

__device__ inline uint32_t convert4(float a, float b, float c, float d, float lo, float hi) {
  v2s w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, lo, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, hi, true);
  return __builtin_bit_cast(uint32_t, w);
}

// 8 values of a row that share a scale.
__device__ inline uint2 convert_row(const float* v, float f) {
  return {convert4(v[0], v[1], v[2], v[3], f, f), convert4(v[4], v[5], v[6], v[7], f, f)};
}

// 8 columns of two rows, each column with its own scale: a conversion takes a column's two rows,
// and a byte permutation sorts them back into rows.
__device__ inline void convert_columns(const float* u, const float* v, const float* f, uint2& a, uint2& b) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = convert4(u[2 * i], v[2 * i], u[2 * i + 1], v[2 * i + 1], f[2 * i], f[2 * i + 1]);
  a = {__builtin_amdgcn_perm(w[1], w[0], 0x06040200), __builtin_amdgcn_perm(w[3], w[2], 0x06040200)};
  b = {__builtin_amdgcn_perm(w[1], w[0], 0x07050301), __builtin_amdgcn_perm(w[3], w[2], 0x07050301)};
}

// ---- the general form

// E4M3 codes of 8 values with one factor each.
__device__ inline uint2 encode8(const float* v, const float* up) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = to_e4m3_range(v[i], up[i]);
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
  return uint2{(uint32_t)a, (uint32_t)b};
}

// The values of 8 E4M3 codes times 2^(s - 127).
__device__ inline Chunk decode8(uint2 w, uint32_t s) {
  // 2^-127 is not a normal number: the product below is exact all the same
  const float f = s ? __uint_as_float(s << 23) : __uint_as_float(1u << 22);
  Chunk c;
  c.v[0] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 0) * f;
  c.v[1] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 1) * f;
  c.v[2] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 2) * f;
  c.v[3] = __builtin_amdgcn_cvt_f32_fp8((int)w.x, 3) * f;
  c.v[4] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 0) * f;
  c.v[5] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 1) * f;
  c.v[6] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 2) * f;
  c.v[7] = __builtin_amdgcn_cvt_f32_fp8((int)w.y, 3) * f;
  return c;
}

}  // namespace mxfp8
