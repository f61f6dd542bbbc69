// Activation functions with 8-bit outputs and an 8-bit checkpoint (mxfp8_act_forward,
// mxfp8_act_backward) on gfx950.
//
// forward:  y = f(u) from the inputs; y leaves in 8 bits in row-wise blocks (the next
//           product), in column-wise blocks (the weight gradient's checkpoint), or rounded to
//           the input type; the inputs leave in 8 bits in row-wise blocks.
// backward: gradients dy * f'(u) at the saved 8-bit inputs, in the same forms.
//
// A SwiGLU forward in BF16 reads 4 and writes 4 bytes per value, backward the same: HBM would need
// 175 us for 8192 x 14336.  The vector units bind it too: 50 instructions per value forward and 64
// backward keep them busy for 88% and 95% of the 207 and 240 us it takes.  One pass: a workgroup owns a 128 x 128 tile,
// so it holds every row-wise and column-wise block it touches whole, keeps the tile's values in
// registers (8 waves: 32 values a thread of each result, which leaves room for 4 waves on a SIMD
// and so for loads in flight), takes the row amax over the 16 lanes that share a row (DPP), the
// column amax over a lane's rows, over the wave's row groups (permlane swaps), then over waves
// through LDS, and writes each output once.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "layer_internal.h"
#include "values.h"

namespace mxfp8 {
namespace {

constexpr int kThreads = 512;
constexpr int kRowsPerPass = 32;  // 8 waves x 4 rows of 16 lanes
constexpr int kPasses = 4;        // 128 rows

struct Mat8 {
  uint8_t* data;
  int64_t ld;
  uint8_t* scale;
  int64_t scale_ld;
};

struct Args {
  int64_t rows, cols;
  const void* in[2];  // forward: the inputs
  int64_t ld_in[2];
  const void* grad;   // backward
  int64_t ld_grad;
  Mat8 saved[2];
  void* out[2];
  int64_t ld_out[2];
  Mat8 row[2], col[2];
  int tiles_c;
};

// s = 1 / (1 + exp(-x)) and c = 1 - s = exp(-x) s, each within a few units in the last place (c
// without the cancellation of 1 - s); below -87.3, where s is under 2^-125, it is taken as 0.  Far
// on the other side c has to reach 0 too: x may be as large as FP32 holds, and x c counts.
struct Sigmoid {
  float s, c;
};
__device__ inline Sigmoid sigmoid(float x) {
  // exp(-x) = 2^t, t = -x log2 e in two parts so that large |x| keeps its relative accuracy
  constexpr float kHi = -1.44269504f, kLo = -1.92596299e-8f;
  const float xc = fminf(fmaxf(x, -87.3f), 150.f);  // 2^t stays finite, and from there on is 0
  const float t = xc * kHi;
  const float r = __builtin_fmaf(xc, kHi, -t) + xc * kLo;
  const float p = __builtin_amdgcn_exp2f(t);
  const float e = __builtin_fmaf(p, r * 0.693147181f, p);
  const float d = 1.f + e;
  const float q = __builtin_amdgcn_rcpf(d);
  const float s = __builtin_fmaf(__builtin_fmaf(-d, q, 1.f), q, q);
  if (x != x) return {x, x};
  return {x < -87.3f ? 0.f : s, x < -87.3f ? 1.f : e * s};
}

constexpr float kGelu = 0.797884561f;  // sqrt(2 / pi)

template <int kFunc>
__device__ inline float apply(float a, float b) {
  if constexpr (kFunc == MXFP8_ACT_NONE) return a;
  if constexpr (kFunc == MXFP8_ACT_GELU) {
    const float z = kGelu * (a + 0.044715f * a * a * a);
    return a * sigmoid(2.f * z).s;
  }
  return a * sigmoid(a).s * b;
}

// Derivatives times d: with respect to a (da) and, for SWIGLU, b (db).
template <int kFunc>
__device__ inline void differentiate(float a, float b, float d, float& da, float& db) {
  if constexpr (kFunc == MXFP8_ACT_GELU) {
    const float z = kGelu * (a + 0.044715f * a * a * a);
    const Sigmoid g = sigmoid(2.f * z);
    const float zp = 2.f * kGelu * (1.f + 3.f * 0.044715f * a * a);
    const float w = g.s * g.c;
    // far out w vanishes faster than anything it is multiplied with, which may be infinite
    da = d * (fabsf(z) > 43.f ? g.s : g.s + a * w * zp);
    db = 0.f;
  } else {
    const Sigmoid g = sigmoid(a);
    da = d * b * (g.s + a * (g.s * g.c));
    db = d * (a * g.s);
  }
}

template <int kCtrl>
__device__ inline uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true));
}

// Over the 16 lanes of a row: quads by permutation, then halves and the row by mirrors.
__device__ inline uint32_t max16(uint32_t v) {
  v = max_dpp<0xB1>(v);   // lane ^ 1
  v = max_dpp<0x4E>(v);   // lane ^ 2
  v = max_dpp<0x141>(v);  // mirror of 8
  return max_dpp<0x140>(v);  // mirror of 16
}

// Over the wave's 4 rows of lanes.
__device__ inline uint32_t max_rows(uint32_t v) {
  auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(p[0], p[1]);
  auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(q[0], q[1]);
}

// Row-wise block of this lane's 16-lane group: scale and codes.
__device__ inline void emit_row(const Mat8& m, const Chunk& c, int64_t r, int64_t col,
                                int64_t valid, bool live) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(c.v[i]));
  a = max16(a);
  uint2 codes;
  if (__any(unusual(a))) {
    a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, finite_bits(c.v[i]));
    a = max16(a);
    const float f = scale_up(scale_of(a));
    const float up[8] = {f, f, f, f, f, f, f, f};
    codes = encode8(c.v, up);
  } else {
    codes = convert_row(c.v, scale_factor(scale_of(a)));
  }
  if (!live) return;
  store8_bytes(m.data, r * m.ld + col, valid, codes);
  if ((threadIdx.x & 15) == 0) m.scale[r * m.scale_ld + col / 128] = (uint8_t)scale_of(a);
}

struct Shared {
  uint32_t part[kThreads / 64][128];
  uint32_t scale[128];
  int unusual;
};

// Column-wise blocks of the tile from the values a thread holds (zero where not live).
__device__ inline void emit_cols(const Mat8& m, const Chunk (&c)[kPasses], Shared& sh, int64_t r0,
                                 int64_t band, int64_t col0, int64_t cols, int64_t rows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t col = col0 + 8 * (tid & 15), valid = cols - col;
  uint32_t a[8], all = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) a[i] = max(a[i], abs_bits(c[p].v[i]));
    all = max(all, a[i]);
  }
  // (also: the shared arrays are free again)
  const bool infinite = __syncthreads_or(all >= kInfinity);
  if (infinite) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = 0;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) a[i] = max(a[i], finite_bits(c[p].v[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max_rows(a[i]);
  if (lane < 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sh.part[wave][8 * lane + i] = a[i];
  }
  if (tid == 0) sh.unusual = infinite;
  __syncthreads();
  if (tid < 128) {
    uint32_t v = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) v = max(v, sh.part[w][tid]);
    const uint32_t s = scale_of(v);
    sh.scale[tid] = s;
    if (unusual(v)) sh.unusual = 1;
    if (col0 + tid < cols) m.scale[band * m.scale_ld + col0 + tid] = (uint8_t)s;
  }
  __syncthreads();
  uint32_t s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = sh.scale[8 * (tid & 15) + i];
  uint2 codes[kPasses];
  if (sh.unusual) {
    float up[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = scale_up(s[i]);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) codes[p] = encode8(c[p].v, up);
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = scale_factor(s[i]);
#pragma unroll
    for (int p = 0; p < kPasses; p += 2)
      convert_columns(c[p].v, c[p + 1].v, f, codes[p], codes[p + 1]);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r < rows && valid > 0) store8_bytes(m.data, r * m.ld + col, valid, codes[p]);
  }
}

template <int kFunc, bool kBF16, bool kBackward>
__global__ __launch_bounds__(kThreads) void act_kernel(const Args g) {
  __shared__ Shared shared;
  saturate_conversions();
  constexpr int kInputs = kFunc == MXFP8_ACT_SWIGLU ? 2 : 1;
  constexpr int kResults = kBackward ? kInputs : 1;
  const int tid = threadIdx.x;
  const int64_t band = blockIdx.x / g.tiles_c;
  const int64_t col0 = int64_t(blockIdx.x % g.tiles_c) * 128, col = col0 + 8 * (tid & 15);
  const int64_t r0 = band * 128 + (tid >> 4);
  const int64_t valid = g.cols - col;
  // all loads first, without a branch where the tile is whole
  Raw<kBF16> in[kBackward ? 1 : kInputs][kPasses];
  uint2 codes[kInputs][kPasses];
  uint32_t scales[kInputs][kPasses];
  auto load = [&](auto whole_) {
    constexpr bool whole = decltype(whole_)::value;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int64_t r = r0 + p * kRowsPerPass;
      const bool live = whole || (r < g.rows && valid > 0);
      const int64_t n = whole ? 8 : live ? valid : 0;
      if constexpr (!kBackward) {
#pragma unroll
        for (int i = 0; i < kInputs; ++i)
          in[i][p] = load_raw<kBF16, true>(g.in[i], live ? r * g.ld_in[i] + col : 0, n);
      } else {
        in[0][p] = load_raw<kBF16, true>(g.grad, live ? r * g.ld_grad + col : 0, n);
#pragma unroll
        for (int i = 0; i < kInputs; ++i) {
          const Mat8& m = g.saved[i];
          codes[i][p] = load8_bytes(m.data, live ? r * m.ld + col : 0, n);
          scales[i][p] = live ? m.scale[r * m.scale_ld + col / 128] : 0;
        }
      }
    }
  };
  if (col0 + 128 <= g.cols && band * 128 + 128 <= g.rows)
    load(std::true_type{});
  else
    load(std::false_type{});
  Chunk y[kResults][kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    const bool live = r < g.rows && valid > 0;
    const int64_t n = live ? valid : 0;
    if constexpr (!kBackward) {
      Chunk u[kInputs];
#pragma unroll
      for (int i = 0; i < kInputs; ++i) u[i] = values_of<kBF16>(in[i][p]);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[0][p].v[e] = apply<kFunc>(u[0].v[e], u[kInputs - 1].v[e]);
      if constexpr (kFunc != MXFP8_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < kInputs; ++i)
          if (g.saved[i].data) emit_row(g.saved[i], u[i], r, col, n, live);
      }
    } else {
      const Chunk d = values_of<kBF16>(in[0][p]);
      Chunk u[kInputs];
#pragma unroll
      for (int i = 0; i < kInputs; ++i) u[i] = decode8(codes[i][p], scales[i][p]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float da, db;
        differentiate<kFunc>(u[0].v[e], u[kInputs - 1].v[e], d.v[e], da, db);
        y[0][p].v[e] = da;
        if constexpr (kResults == 2) y[1][p].v[e] = db;
      }
    }
#pragma unroll
    for (int o = 0; o < kResults; ++o) {
      if (live && g.out[o]) store8<kBF16>(g.out[o], r * g.ld_out[o] + col, n, y[o][p]);
      if (g.row[o].data) emit_row(g.row[o], y[o][p], r, col, n, live);
    }
  }
#pragma unroll
  for (int o = 0; o < kResults; ++o)
    if (g.col[o].data) emit_cols(g.col[o], y[o], shared, r0, band, col0, g.cols, g.rows);
}

Mat8 mat(const mxfp8_mat8& m) {
  return {static_cast<uint8_t*>(m.data), m.ld, static_cast<uint8_t*>(m.scale), m.scale_ld};
}

Args args_of(const mxfp8_act& a) {
  Args g{};
  g.rows = a.rows;
  g.cols = a.cols;
  for (int i = 0; i < 2; ++i) {
    g.in[i] = a.input[i].ptr;
    g.ld_in[i] = a.input[i].ld;
    g.saved[i] = mat(a.saved[i]);
    g.out[i] = a.out[i].ptr;
    g.ld_out[i] = a.out[i].ld;
    g.row[i] = mat(a.row[i]);
    g.col[i] = mat(a.col[i]);
  }
  g.grad = a.grad.ptr;
  g.ld_grad = a.grad.ld;
  g.tiles_c = (int)((a.cols + 127) / 128);
  return g;
}

template <int kFunc, bool kBackward>
hipError_t launch(const mxfp8_act& a, hipStream_t s) {
  const Args g = args_of(a);
  const dim3 grid((unsigned)((a.rows + 127) / 128 * g.tiles_c));
  if (a.dtype == MXFP8_BF16)
    act_kernel<kFunc, true, kBackward><<<grid, kThreads, 0, s>>>(g);
  else
    act_kernel<kFunc, false, kBackward><<<grid, kThreads, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act_forward(const mxfp8_act& a, hipStream_t s) {
  if (a.func == MXFP8_ACT_NONE) return launch<MXFP8_ACT_NONE, false>(a, s);
  if (a.func == MXFP8_ACT_GELU) return launch<MXFP8_ACT_GELU, false>(a, s);
  return launch<MXFP8_ACT_SWIGLU, false>(a, s);
}

hipError_t launch_act_backward(const mxfp8_act& a, hipStream_t s) {
  if (a.func == MXFP8_ACT_GELU) return launch<MXFP8_ACT_GELU, true>(a, s);
  return launch<MXFP8_ACT_SWIGLU, true>(a, s);
}

}  // namespace mxfp8
