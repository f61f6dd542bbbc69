// Products of 8-bit matrices with block scales on gfx950 (mxfp8_matmul).
//
//   out[m][n] = round(sum_k a(m, k) b(n, k) + addend[m][n]),  a(m, k) = code * 2^(scale - 127)
//
// plan_product (layer_plan.cpp) picks the kernel: product_few.hip for a few tokens,
// product_large.h for operands in aligned rows, and here, for rows at any alignment, a plain
// kernel: a workgroup computes one tile, walking the sum in steps of 128 values whose codes pass
// through registers into two LDS buffers in turn.  333 x 1001 x 4095 in FP32 takes 28 us, bound by
// the latency of those loads with 4 steps a workgroup.
//
// Two arithmetics:
//  - BF16 output: v_mfma_scale_f32_32x32x64_f8f6f4 on the codes, E8M0 scales applied by the
//    matrix unit (4.1 PFLOP/s measured in registers).  The unit aligns the products of
//    each 8 successive values to the largest of them and drops what lies below 2^-13 of it
//    (measured; from one such 8 to the next it keeps 2^-23): 1.4e-5 of the result's norm on
//    random data, against 1.7e-3 of the rounding to BF16.
//  - FP32 output (kExact): codes become BF16 exactly (v_cvt_scalef32_pk_bf16_fp8, which also
//    applies the scale) and v_mfma_f32_32x32x16_bf16 sums them in FP32: 1e-7 of the norm,
//    at half the matrix rate (2.1 PFLOP/s measured in registers).
//
// The sum's order is free as long as both operands agree, so lane l of a wave holds, for row
// l % 32 of its 32-row fragment and each 32-value block q of the step, the 16 values starting
// at 32 q + 16 (l / 32).  That is the order in which the scaled instruction pairs values with
// scales: its registers 0-3 hold the first 32-value block of 64, registers 4-7 the second, and
// lane half h supplies the scale of block h.
#include "product_device.h"

namespace mxfp8 {
namespace {

// ---------------------------------------------------------------- LDS tiles
//
// A tile holds T outer values x 128 of the sum as 16-byte chunks.  ALONG_COLS: [T rows][8
// chunks], chunk c of row r stored at position c ^ ((r >> 1) & 7), so that 16 lanes reading
// one chunk of 16 successive rows touch all 64 banks once.  ALONG_ROWS: [128 k][T / 16
// chunks], chunk c of row k at position c ^ f(k), f even, so that the 16 8-byte reads that a
// half wave makes of 8 rows x 2 neighbouring chunks do the same; ds_read_b64_tr_b8 then turns
// 8 rows x 16 columns of bytes into 8 successive k for each of 16 lanes.

// Chunk of the tile that goes to 16-byte slot `slot`: its outer offset (the row, or the first
// of 16 columns) and its offset along the sum.
template <int T, bool kRows>
__device__ inline void slot_chunk(int slot, int& outer, int& kk) {
  if constexpr (kRows) {
    constexpr int chunks = T / 16;
    kk = slot / chunks;
    outer = 16 * ((slot % chunks) ^ rows_swizzle<T>(kk));
  } else {
    outer = slot / 8;
    kk = 16 * ((slot % 8) ^ ((outer >> 1) & 7));
  }
}

// 16 bytes at p of which the first `valid` exist; the rest become 0.
__device__ inline v4i load_chunk(const uint8_t* p, int64_t valid) {
  v4i v = {0, 0, 0, 0};
  if (valid >= 16) {
    __builtin_memcpy(&v, p, 16);  // any alignment
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < valid) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    v = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
  }
  return v;
}

// Fills one tile buffer of an operand by way of registers.  Values past the array's end are 0.
template <int T, bool kRows, int kThreads>
struct Filler {
  static constexpr int kPer = T * 8 / kThreads;
  static_assert(T * 8 % kThreads == 0, "whole chunks per thread");
  v4i reg[kPer];

  __device__ inline void load(const Operand& o, int64_t outer0, int64_t k, int64_t k0, int tid) {
    // Whole chunks throughout (rows past the end repeat the last one: they are not stored): no
    // branch between the loads.
    if (k0 + kStep <= k && (!kRows || outer0 + T <= o.outer)) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        int outer, kk;
        slot_chunk<T, kRows>(i * kThreads + tid, outer, kk);
        int64_t x = outer0 + outer;
        if constexpr (!kRows) x = x < o.outer ? x : o.outer - 1;
        const uint8_t* p = kRows ? o.data + (k0 + kk) * o.ld + x : o.data + x * o.ld + k0 + kk;
        __builtin_memcpy(&reg[i], p, 16);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      int outer, kk;
      slot_chunk<T, kRows>(i * kThreads + tid, outer, kk);
      int64_t valid;
      const uint8_t* p;
      if constexpr (kRows) {
        valid = k0 + kk < k ? o.outer - (outer0 + outer) : 0;
        p = o.data + (k0 + kk) * o.ld + outer0 + outer;
      } else {
        valid = outer0 + outer < o.outer ? k - (k0 + kk) : 0;
        p = o.data + (outer0 + outer) * o.ld + k0 + kk;
      }
      reg[i] = load_chunk(p, valid);
    }
  }

  __device__ inline void store(uint8_t* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      *reinterpret_cast<v4i*>(lds + 16 * (i * kThreads + tid)) = reg[i];
  }
};

// The 16 codes of a lane for fragment rows outer0 .. outer0 + 31 and 32-value block q.
template <int T, bool kRows>
__device__ inline v4i read_codes(const uint8_t* lds, int outer0, int q, int lane) {
  const int h = lane >> 5;
  if constexpr (kRows) {
    const int i = lane & 15, k = 32 * q + 16 * h + (i >> 1);
    const int c = (outer0 >> 4) + ((lane >> 4) & 1);
    const uint8_t* p = lds + k * T + 16 * (c ^ rows_swizzle<T>(i >> 1)) + 8 * (i & 1);
    auto* lp = LDS_PTR(v2i, const_cast<uint8_t*>(p));
    const v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32(lp);
    const v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32(lp + T);  // 8 rows on
    return v4i{lo[0], lo[1], hi[0], hi[1]};
  } else {
    const int r = lane & 31;
    return *reinterpret_cast<const v4i*>(lds + (outer0 + r) * 128 +
                                         16 * ((2 * q + h) ^ ((r >> 1) & 7)));
  }
}

// ---------------------------------------------------------------- the kernel

// Tile TM x TN on WM x WN waves.
template <int TM, int TN, int WM, int WN, bool kARows, bool kBRows, bool kExact>
__global__ __launch_bounds__(WM* WN * 64, 2) void product_kernel(const ProductArgs g) {
  constexpr int kThreads = WM * WN * 64;
  constexpr int FM = TM / WM / 32, FN = TN / WN / 32;  // 32 x 32 fragments of a wave
  __shared__ __attribute__((aligned(16))) uint8_t sa[2][TM * 128], sb[2][TN * 128];
  __shared__ __attribute__((aligned(16))) v4i ss[2][TM + TN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave / WN) * (TM / WM), wn = (wave % WN) * (TN / WN);

  const int tile = blockIdx.x;
  const int64_t m0 = int64_t(tile % g.tiles_m) * TM, n0 = int64_t(tile / g.tiles_m) * TN;
  const int64_t total = (g.k + kStep - 1) / kStep;
  const int64_t first = int64_t(blockIdx.y) * g.steps;
  const int64_t last = first + g.steps < total ? first + g.steps : total;

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int t = 0; t < 16; ++t) acc[i][j][t] = 0.f;

  Filler<TM, kARows, kThreads> fa;
  Filler<TN, kBRows, kThreads> fb;
  constexpr int kRowsPer = (TM + TN + kThreads - 1) / kThreads;
  ScaleBytes sc[kRowsPer];
  auto fetch_scales = [&](int64_t group) {
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const int r = i * kThreads + tid;
      if (r < TM)
        sc[i] = load_scales(g.a, m0 + r, g.k, group);
      else if (r < TM + TN)
        sc[i] = load_scales(g.b, n0 + r - TM, g.k, group);
    }
  };
  auto stage_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const int r = i * kThreads + tid;
      if (r < TM + TN)
        ss[buf][r] = arrange_scales(sc[i], r < TM ? g.a.block_shift : g.b.block_shift);
    }
  };

  if (first < last) {
    fa.load(g.a, m0, g.k, first * kStep, tid);
    fb.load(g.b, n0, g.k, first * kStep, tid);
    fetch_scales(first / kGroup);
    stage_scales(0);
    fa.store(sa[0], tid);
    fb.store(sb[0], tid);
  }
  v4i da[FM], db[FN];
  for (int64_t s = first; s < last; ++s) {
    const int buf = (int)(s - first) & 1, sub = (int)s & 3;
    const int sbuf = (int)((s - first) / kGroup) & 1;  // first is a multiple of kGroup
    // this wave's part of step s is written; then everyone's is, and everyone has read s - 1
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier();
    if (s + 1 < last) {
      fa.load(g.a, m0, g.k, (s + 1) * kStep, tid);
      fb.load(g.b, n0, g.k, (s + 1) * kStep, tid);
    }
    if (sub == 0) {
      if (s + kGroup < last) fetch_scales(s / kGroup + 1);
#pragma unroll
      for (int i = 0; i < FM; ++i) da[i] = ss[sbuf][wm + 32 * i + (lane & 31)];
#pragma unroll
      for (int j = 0; j < FN; ++j) db[j] = ss[sbuf][TM + wn + 32 * j + (lane & 31)];
    }
    const uint8_t* ta = sa[buf];
    const uint8_t* tb = sb[buf];
    if constexpr (!kExact) {
      const int h = lane >> 5;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        v8i a[FM], b[FN];
        int ea[FM], eb[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v4i lo = read_codes<TN, kBRows>(tb, wn + 32 * j, 2 * kk, lane);
          const v4i hi = read_codes<TN, kBRows>(tb, wn + 32 * j, 2 * kk + 1, lane);
          b[j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          eb[j] = (h ? db[j][2 * kk + 1] : db[j][2 * kk]) >> (8 * sub);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const v4i lo = read_codes<TM, kARows>(ta, wm + 32 * i, 2 * kk, lane);
          const v4i hi = read_codes<TM, kARows>(ta, wm + 32 * i, 2 * kk + 1, lane);
          a[i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          ea[i] = (h ? da[i][2 * kk + 1] : da[i][2 * kk]) >> (8 * sub);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                a[i], b[j], acc[i][j], 0, 0, 0, ea[i], 0, eb[j]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v8b a[FM][2], b[FN][2];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const v4i c = read_codes<TN, kBRows>(tb, wn + 32 * j, q, lane);
          const float e = __int_as_float(((db[j][q] >> (8 * sub)) & 0xFF) << 23);
          b[j][0] = to_bf16(c[0], c[1], e);
          b[j][1] = to_bf16(c[2], c[3], e);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const v4i c = read_codes<TM, kARows>(ta, wm + 32 * i, q, lane);
          const float e = __int_as_float(((da[i][q] >> (8 * sub)) & 0xFF) << 23);
          a[i][0] = to_bf16(c[0], c[1], e);
          a[i][1] = to_bf16(c[2], c[3], e);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i][t], b[j][t], acc[i][j],
                                                                  0, 0, 0);
      }
    }
    if (s + 1 < last) {
      fa.store(sa[buf ^ 1], tid);
      fb.store(sb[buf ^ 1], tid);
    }
    if (sub == 3 && s + 1 < last) stage_scales(sbuf ^ 1);
  }
  // The accumulators are read by ordinary instructions from here on: let the last matrix
  // instructions retire (16 passes) before that.
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("s_nop 15\n\ts_nop 7" : "+v"(acc[i][j]));

  // Lane l holds column n = l % 32 of a fragment, and 4 of each 8 of its rows m: a store covers 32
  // neighbouring outputs of two rows.
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t n = n0 + wn + 32 * j + (lane & 31);
    if (n >= g.n) continue;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const int64_t m = m0 + wm + 32 * i + 8 * (t / 4) + 4 * (lane >> 5) + t % 4;
        if (m >= g.m) continue;
        float v = acc[i][j][t];
        if (g.part) {
          g.part[(int64_t(blockIdx.y) * g.m + m) * g.n + n] = v;
        } else {
          if (g.add) v += g.add[m * g.ldadd + n];
          if constexpr (kExact)
            static_cast<float*>(g.out)[m * g.ldo + n] = v;
          else
            static_cast<uint16_t*>(g.out)[m * g.ldo + n] = bf16_bits(v);
        }
      }
  }
}

// Joins the parts of a split sum in their order, adds the addend and rounds.
template <bool kF32>
__global__ __launch_bounds__(256) void join_kernel(const ProductArgs g, int splits) {
  const int64_t mn = g.m * g.n;
  for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < mn; e += int64_t(gridDim.x) * 256) {
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += g.part[s * mn + e];
    const int64_t m = e / g.n, n = e % g.n;
    if (g.add) v += g.add[m * g.ldadd + n];
    if constexpr (kF32)
      static_cast<float*>(g.out)[m * g.ldo + n] = v;
    else
      static_cast<uint16_t*>(g.out)[m * g.ldo + n] = bf16_bits(v);
  }
}

template <int TM, int TN, int WM, int WN, bool kExact>
void launch_kind(const ProductArgs& g, bool ar, bool br, dim3 grid, hipStream_t s) {
  const dim3 block(WM * WN * 64);
  if (ar && br)
    product_kernel<TM, TN, WM, WN, true, true, kExact><<<grid, block, 0, s>>>(g);
  else if (ar)
    product_kernel<TM, TN, WM, WN, true, false, kExact><<<grid, block, 0, s>>>(g);
  else if (br)
    product_kernel<TM, TN, WM, WN, false, true, kExact><<<grid, block, 0, s>>>(g);
  else
    product_kernel<TM, TN, WM, WN, false, false, kExact><<<grid, block, 0, s>>>(g);
}

Operand operand_of(const mxfp8_operand& o, int64_t outer) {
  Operand r;
  r.data = static_cast<const uint8_t*>(o.data);
  r.scale = static_cast<const uint8_t*>(o.scale);
  r.ld = o.ld;
  r.outer = outer;
  r.s_outer = o.along == MXFP8_ALONG_COLS ? o.scale_ld : 1;
  r.s_block = o.along == MXFP8_ALONG_COLS ? 1 : o.scale_ld;
  r.across_shift = o.across == 128 ? 7 : 0;
  r.block_shift = o.block == 128 ? 2 : 0;
  return r;
}

}  // namespace

hipError_t launch_product(const mxfp8_product& p, const ProductPlan& plan, hipStream_t s) {
  ProductArgs g{};
  g.a = operand_of(p.a, p.m);
  g.b = operand_of(p.b, p.n);
  g.m = p.m;
  g.n = p.n;
  g.k = p.k;
  g.out = p.out.ptr;
  g.ldo = p.out.ld;
  g.add = static_cast<const float*>(p.addend.ptr);
  g.ldadd = p.addend.ld;
  g.part = plan.join ? static_cast<float*>(p.workspace) : nullptr;
  g.steps = plan.steps;
  g.packed = plan.packed ? static_cast<uint8_t*>(p.workspace) : nullptr;
  if (g.part) g.part += plan.packed / 4;
  g.tiles_m = (int)((p.m + plan.tile_m - 1) / plan.tile_m);
  g.tiles_n = (int)((p.n + plan.tile_n - 1) / plan.tile_n);
  const dim3 grid((unsigned)g.tiles_m * (unsigned)g.tiles_n, (unsigned)plan.splits);
  const bool ar = p.a.along == MXFP8_ALONG_ROWS, br = p.b.along == MXFP8_ALONG_ROWS;
  const bool f32 = p.out_dtype == MXFP8_FP32;
  hipError_t e = hipSuccess;
  if (plan.variant == kFew) {
    e = launch_few(g, f32, s);
  } else if (plan.variant == kLarge) {
    e = launch_large_product(g, plan, ar, br, f32, s);
  } else if (plan.variant == kTile128) {
    if (f32)
      launch_kind<128, 128, 2, 2, true>(g, ar, br, grid, s);
    else
      launch_kind<128, 128, 2, 2, false>(g, ar, br, grid, s);
  } else {
    if (f32)
      launch_kind<32, 128, 1, 4, true>(g, ar, br, grid, s);
    else
      launch_kind<32, 128, 1, 4, false>(g, ar, br, grid, s);
  }
  if (e == hipSuccess) e = hipGetLastError();
  if (e != hipSuccess || !plan.join) return e;
  const int64_t want = (p.m * p.n + 255) / 256;
  const dim3 jgrid((unsigned)(want < 4096 ? want : 4096));
  if (f32)
    join_kernel<true><<<jgrid, 256, 0, s>>>(g, plan.splits);
  else
    join_kernel<false><<<jgrid, 256, 0, s>>>(g, plan.splits);
  return hipGetLastError();
}

}  // namespace mxfp8
