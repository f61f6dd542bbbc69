// The matrix product's main kernel, for operands whose 16-byte chunks go straight to LDS
// (plan_product's `direct`); included by one file for each tile size.  See product.hip for the
// arithmetic.
//
// 4 waves of 2 x 2 share a TM x TN tile, a wave holding FM x FN fragments of 32 x 32 in
// accumulator registers: 128 x 128 a wave for 256 x 256, so that a wave reads 16 KB of codes
// from LDS per half step of 64 values for 16 scaled instructions of 64 cycles (8 waves of
// 128 x 64 would read half as much again).
//
// The sum runs in half steps of 64 values through a ring of 4 LDS buffers.  In the phase of half
// t a wave multiplies the fragments of half t, which it holds in registers, reads the fragments
// of half t + 1 into its other register set, and starts the loads of half t + 4 into the buffer
// of half t, which every wave has read.  One LDS read, and every other time one load, follow
// each matrix instruction: bunched, they hold up the instructions behind them.  A phase ends
// with this wave's loads of half t + 2 landed (the two phases' worth after them stay in flight)
// and a barrier, so a load has two to three phases to land, 2048 to 3072 matrix cycles for
// 256 x 256.  Two buffers of whole steps, whose loads fetch full 128-byte lines, leave it one to
// two phases: 8192 x 14336 x 4096 took 515 us so, and 448 us with the ring
// (the same inputs every call; the kernel as it is takes 443 us so, and 461 with inputs that change).  The 256 x 256 instances spill 20 to
// 28 registers in BF16 and 66 to 112 in FP32, outside the main loop but for one: FP32 with only b
// ALONG_ROWS reloads three in four half steps.
//
// The workgroups stay for all their tiles (one per CU), and the ring runs on from one tile into
// the next: while a tile is stored, the first halves of the next land.
//
// Scales come packed by pack_scales_kernel, 16 bytes for each row and group of 512 values of
// the sum, whatever their layout was: the loads of a group are one 16-byte load per row, and a
// lane finds its byte at a fixed place.  Rows and blocks past the end repeat the last ones: such
// rows are not stored, such blocks' codes are 0.
#pragma once

#include <type_traits>

#include "product_device.h"

namespace mxfp8 {
namespace {

template <int v>
using Const = std::integral_constant<int, v>;

// f(Const<0>), ..., f(Const<N - 1>): a loop whose index is a constant in its body.
template <int N, typename Body>
__device__ inline void each(Body&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(Const<N - 1>{});
  }
}

// One operand's loads; load_bounds.h has their addresses.  LDS layout of a half: ALONG_COLS [T
// rows][4 chunks of 16], chunk c of row r at position c ^ ((r >> 2) & 3); ALONG_ROWS [64 k][T / 16
// chunks], chunk c of row k at c ^ rows_swizzle(k).  16 lanes reading one chunk of 16 successive
// rows, or 8 rows of 2 neighbouring chunks, so touch every bank once.
template <int T, bool kRows>
struct Stream {
  static constexpr int kLoads = T / 64;  // 16-byte loads of a thread per half
  static constexpr int kBytes = T * kHalf;
  uint32_t off[kLoads];  // of the thread's chunks from the half's base
  int kk;                // ALONG_COLS: where they lie in the half
  const uint8_t* base;
  uint32_t extent;       // ALONG_COLS: bytes the loads may touch; ALONG_ROWS: columns from outer0 on
  int left;              // values of the sum from the half's start

  __device__ inline void init(const Operand& o, int tid) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const Place p = place_of<T, kRows>(i * 256 + tid);
      off[i] = (uint32_t)(p.row * (int)o.ld + p.at);
      kk = kRows ? 0 : p.at;  // the same for every i
    }
  }

  // From values k0 .. kend - 1 of the sum on, for outer values from outer0 on.
  __device__ inline void start(const Operand& o, int64_t outer0, int64_t k0, int64_t kend) {
    left = (int)(kend - k0);
    if constexpr (kRows) {
      base = o.data + k0 * o.ld + outer0;
      extent = (uint32_t)(o.outer - outer0);
    } else {
      base = o.data + outer0 * o.ld + k0;
      extent = cols_extent<T>(o.outer - outer0, o.ld);
    }
  }
  __device__ inline void finish() { left = 0; }  // nothing more: every load reads 0

  // The half's buffer resource: lanes past the last row read 0.
  __device__ inline v4i resource(const Operand& o) const {
    const uint64_t b = (uint64_t)base;
    const uint32_t e = kRows ? rows_extent(left, (int)o.ld, extent) : extent;
    return v4i{__builtin_amdgcn_readfirstlane((int)b),
               __builtin_amdgcn_readfirstlane((int)(b >> 32) & 0xFFFF),
               __builtin_amdgcn_readfirstlane((int)e), 0x00020000};
  }

  // Starts load i of the half into LDS at byte `lds` (the buffer plus 1 KB per wave).
  __device__ inline void load(int i, const v4i& rsrc, uint32_t lds) const {
    uint32_t o = off[i];
    if constexpr (!kRows) o = cols_offset(o, kk, left);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds + i * 4096), "v"(o), "s"(rsrc));
  }

  __device__ inline void next(const Operand& o) {
    const int64_t advance = kRows ? kHalf * o.ld : kHalf;
    base += advance;
    left -= kHalf;
  }
};

// Where a lane reads its codes of 32-value block b of a half, for fragments of 32 outer values
// from outer0 on.
template <int T, bool kRows, int F>
struct Reader {
  uint32_t at[kRows ? F : 2];

  __device__ inline void init(uint32_t lds, int outer0, int lane) {
    const int h = lane >> 5;
    if constexpr (kRows) {
      const int i = lane & 15, k = 16 * h + (i >> 1);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int c = ((outer0 + 32 * f) >> 4) + ((lane >> 4) & 1);
        at[f] = lds + k * T + 16 * (c ^ rows_swizzle<T>(i >> 1)) + 8 * (i & 1);
      }
    } else {
      const int r = lane & 31;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        at[b] = lds + (outer0 + r) * kHalf + 16 * ((2 * b + h) ^ ((r >> 2) & 3));
    }
  }

  __device__ inline v4i read(int slot, int f, int b) const {
    if constexpr (kRows) {
      auto* p = LDS_AT(v2i, at[f] + slot * (T * kHalf) + b * (32 * T));
      const v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32(p);
      const v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32(p + T);  // 8 rows on
      return v4i{lo[0], lo[1], hi[0], hi[1]};
    } else {
      auto* p = LDS_AT(v4i, at[b] + slot * (T * kHalf) + f * (32 * kHalf));
      return *p;
    }
  }
};

// Before loads read buffer resources that a vector instruction may have written: 5 wait states.
__device__ inline void settle(v4i& a, v4i& b) { asm volatile("s_nop 4" : "+s"(a), "+s"(b)); }

// Operand of s_waitcnt: at most vm loads and stores, and lgkm LDS operations, in flight.
constexpr int wait_code(int vm, int lgkm) {
  return (vm & 15) | (vm >> 4) << 14 | 7 << 4 | lgkm << 8;
}

template <bool kF32>
struct Out;
template <>
struct Out<false> {
  typedef uint16_t type;
  static constexpr int kPer = 8;  // values of a 16-byte store
  __device__ static inline type round(float v) { return bf16_bits(v); }
};
template <>
struct Out<true> {
  typedef float type;
  static constexpr int kPer = 4;
  __device__ static inline type round(float v) { return v; }
};

// Stores a wave's FM x FN fragments through kStage bytes of LDS of its own, so that a store covers whole
// rows of the wave's columns, 16 bytes a lane.  16-byte chunk c of staged row r lies at position
// c ^ r (BF16) or c ^ 2 r (FP32): conflict-free both ways.  `add` is for FP32 only: a BF16 output
// with an addend goes through FP32 partial sums and join_kernel, since code for it here costs
// every BF16 tile registers (8192 x 14336 x 4096, the same inputs every call: 486 us
// instead of 444).
template <bool kF32, int kStage, int FM, int FN>
__device__ inline void store_tile(v16f (&acc)[FM][FN], uint8_t* lds, int64_t m0, int64_t n0, int64_t m,
                                  int64_t n, void* out, int64_t ldo, const float* add,
                                  int64_t ldadd, int lane) {
  typedef typename Out<kF32>::type T;
  constexpr int kPer = Out<kF32>::kPer;          // values of a chunk
  constexpr int kCols = 32 * FN;
  constexpr int kChunks = kF32 ? 32 : 16;        // positions of a staged row
  constexpr int kRows = kStage / (16 * kChunks);   // rows staged at a time
  constexpr int kStore = 64 / kChunks;           // rows of one store
  const int mine = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    // keeps the accumulators where they are until their turn
#pragma unroll
    for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
    for (int part = 0; part < 32 / kRows; ++part) {
      const int64_t row0 = m0 + 32 * i + part * kRows;
      if (mine / kRows == part) {
        const int r = mine % kRows;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            T v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = Out<kF32>::round(acc[i][j][4 * t + e]);
            const int c = kF32 ? (8 * j + 2 * t + h) ^ (2 * r) : (4 * j + t) ^ r;
            __builtin_memcpy(lds + r * (16 * kChunks) + 16 * c + (kF32 ? 0 : 8 * h), v, sizeof v);
          }
      }
      asm volatile("" ::: "memory");
#pragma unroll
      for (int p = 0; p < kRows / kStore; ++p) {
        const int r = p * kStore + lane / kChunks, c = lane % kChunks;
        T v[kPer];
        __builtin_memcpy(v, lds + r * (16 * kChunks) + 16 * (kF32 ? c ^ (2 * r) : c ^ r), 16);
        const int64_t row = row0 + r, col = n0 + c * kPer;
        if (row < m && col < n && c * kPer < kCols) {
          T* o = static_cast<T*>(out) + row * ldo + col;
          if (col + kPer <= n) {
            if constexpr (kF32) {
              if (add) {
                float x[4];
                __builtin_memcpy(x, add + row * ldadd + col, 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += x[e];
              }
            }
            __builtin_memcpy(o, v, 16);
          } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
              if (col + e < n) {
                if constexpr (kF32) {
                  if (add) v[e] += add[row * ldadd + col + e];
                }
                o[e] = v[e];
              }
          }
        }
      }
      asm volatile("" ::: "memory");
    }
  }
}

// Workgroups of a CU: a 256-wide tile takes all its LDS.
constexpr int resident(int tm, int tn) { return tm + tn > 256 ? 1 : 2; }

template <int TM, int TN, bool kARows, bool kBRows, bool kExact>
__global__ __launch_bounds__(256, resident(TM, TN)) void large_kernel(const ProductArgs g, int units) {
  constexpr int FM = TM / 64, FN = TN / 64, F = FM + FN;
  typedef Stream<TM, kARows> StreamA;
  typedef Stream<TN, kBRows> StreamB;
  constexpr int kLoads = StreamA::kLoads + StreamB::kLoads;
  constexpr int kRing = 4 * (StreamA::kBytes + StreamB::kBytes);
  constexpr int kScaleBytes = (TM + TN) * 16;
  constexpr int kStage = resident(TM, TN) == 1 ? 4096 : 2048;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing + 2 * kScaleBytes + 4 * kStage];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * (TM / 2), wn = (wave & 1) * (TN / 2);
  const uint32_t lds0 = (uint32_t)(uintptr_t)LDS_PTR(uint8_t, lds);
  const uint32_t ldsb = lds0 + 4 * StreamA::kBytes, ldss = lds0 + kRing, wlds = 1024 * wave;

  // A unit of work is a tile, or a part of its sum: whole groups of 4 steps.
  const int all = (int)((g.k + kStep - 1) / kStep), groups = (all + kGroup - 1) / kGroup;
  struct Unit {
    int64_t m0, n0, k0, kend;
    int part, halves, group0;  // halves: a multiple of 4 (zeros past the end)
  };
  auto unit_of = [&](int id) {
    Unit u;
    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n;
    u.part = id / tiles;
    tile_of(id - u.part * tiles, g.tiles_m, g.tiles_n, tm, tn);
    u.m0 = int64_t(tm) * TM;
    u.n0 = int64_t(tn) * TN;
    const int first = u.part * (int)g.steps, steps = min((int)g.steps, all - first);
    u.group0 = first / kGroup;
    u.k0 = int64_t(first) * kStep;
    u.kend = u.k0 + int64_t(steps) * kStep < g.k ? u.k0 + int64_t(steps) * kStep : g.k;
    u.halves = (2 * steps + 3) & ~3;
    return u;
  };

  StreamA la;
  StreamB lb;
  la.init(g.a, tid);
  lb.init(g.b, tid);
  Reader<TM, kARows, FM> ra;
  Reader<TN, kBRows, FN> rb;
  ra.init(lds0, wm, lane);
  rb.init(ldsb, wn, lane);

  // Scales: this wave's 64 rows of each operand for a group, into one of two buffers in turn.
  const int wa = wave % (TM / 64), wb = wave % (TN / 64);
  const uint8_t* pa = g.packed + (64 * wa + lane) * 16;
  const uint8_t* pb = g.packed + (int64_t(groups) * g.tiles_m * TM + 64 * wb + lane) * 16;
  const int64_t ga = int64_t(g.tiles_m) * TM, gb = int64_t(g.tiles_n) * TN;
  auto load_group = [&](const Unit& u, int group, int buf) {
    const int gr = min(u.group0 + group, groups - 1);
    const uint32_t dst = ldss + buf * kScaleBytes;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(dst + 1024 * wa), "v"(pa + (gr * ga + u.m0) * 16));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(dst + TM * 16 + 1024 * wb), "v"(pb + (gr * gb + u.n0) * 16));
  };
  auto load_half = [&](int i, const v4i& qa, const v4i& qb, int slot) {
    if (i < StreamA::kLoads)
      la.load(i, qa, lds0 + slot * StreamA::kBytes + wlds);
    else
      lb.load(i - StreamA::kLoads, qb, ldsb + slot * StreamB::kBytes + wlds);
  };

  v16f acc[FM][FN];
  // No instruction: keeps a phase's matrix instructions on its side of the barrier.
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  // fragments (FN of b, then FM of a) of two halves, two 32-value blocks each
  v4i fr[2][F][2];
  auto read_block = [&](int set, int f, int b, int slot) {
    fr[set][f][b] = f < FN ? rb.read(slot, f, b) : ra.read(slot, f - FN, b);
  };
  // Scales of the group in registers.  pack_scales_kernel orders a row's 16 bytes as dwords
  // [block 0][block 2][block 1][block 3] of each step, byte s of a dword being step s's.  Scaled
  // instructions: lane half h needs blocks h and 2 + h (half steps 0 and 1).  Exact: all four.
  typedef typename std::conditional<kExact, v4i, v2i>::type Scales;
  Scales group_sc[F];
  const uint32_t srow = ldss + 16 * (lane & 31) + (kExact ? 0 : 8 * h);
  auto read_group = [&](int buf) {
#pragma unroll
    for (int f = 0; f < F; ++f)
      group_sc[f] = *LDS_AT(Scales, srow + buf * kScaleBytes +
                                        16 * (f < FN ? TM + wn + 32 * f : wm + 32 * (f - FN)));
  };
  // Scale operands of a half's scaled instructions, or scale factors of its blocks.
  int sc[2][F];
  auto set_scale = [&](int into, int half, int block, int t, int f) {  // half t = .. `half` mod 2
    const int shift = 8 * ((t >> 1) & 3);
    if constexpr (kExact)
      sc[into][f] = ((group_sc[f][half + 2 * block] >> shift) & 0xFF) << 23;
    else
      sc[into][f] = group_sc[f][half] >> shift;
  };

  v8b bf[2][F];  // kExact: 8 values of each fragment in BF16, of this round and the next
  auto convert = [&](int set, int f, int u) {  // round u: half of block u / 2
    const float e = __int_as_float(sc[u >> 1][f]);
    const v4i c = fr[set][f][u >> 1];
    bf[u & 1][f] = (u & 1) ? to_bf16(c[2], c[3], e) : to_bf16(c[0], c[1], e);
  };

  // Phase of half t of the unit, whose fragments are in set slot & 1; t1: the next half's place
  // in its unit.
  constexpr int kMul = FM * FN, kReads = 2 * F;
  constexpr int kAll = (kExact ? 4 : 1) * kMul;  // matrix instructions of a phase
  constexpr int kLead = kAll > 2 ? 2 : 1;        // .. before its first load
  auto phase = [&](auto slot_, int t, int t1, int scale_buf) {
    constexpr int slot = decltype(slot_)::value, set = slot & 1;
    v4i qa, qb;
    each<kAll>([&](auto at_) {
      constexpr int at = decltype(at_)::value, u = at / kMul, n = at % kMul, i = n / FN, j = n % FN;
      if constexpr (!kExact) {
        const v4i bl = fr[set][j][0], bh = fr[set][j][1];
        const v4i al = fr[set][FN + i][0], ah = fr[set][FN + i][1];
        const v8i b = {bl[0], bl[1], bl[2], bl[3], bh[0], bh[1], bh[2], bh[3]};
        const v8i a = {al[0], al[1], al[2], al[3], ah[0], ah[1], ah[2], ah[3]};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            b, a, acc[i][j], 0, 0, 0, sc[set][j], 0, sc[set][FN + i]);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[u & 1][j], bf[u & 1][FN + i],
                                                            acc[i][j], 0, 0, 0);
      }
      if constexpr (at == 0 && slot == 3) read_group(scale_buf);  // the group of the next half
      if constexpr (at == 1) {
        qa = la.resource(g.a);
        qb = lb.resource(g.b);
        settle(qa, qb);
      }
      each<kReads>([&](auto r_) {
        constexpr int r = decltype(r_)::value;
        // scaled: over the whole phase; exact: in its first two rounds, before the last converts
        // the first of them
        if constexpr (r * (kExact ? kAll / 2 : kAll) / kReads == at)
          read_block(set ^ 1, r / 2, r % 2, (slot + 1) & 3);
      });
      each<kLoads>([&](auto l_) {
        constexpr int l = decltype(l_)::value;
        if constexpr (kLead + l * (kAll - kLead) / kLoads == at) load_half(l, qa, qb, slot);
      });
      each<F>([&](auto f_) {
        constexpr int f = decltype(f_)::value;
        if constexpr (!kExact) {  // the next phase's scales
          if constexpr (kAll / 2 + f * kAll / (2 * F) == at) set_scale(set ^ 1, set ^ 1, 0, t1, f);
        } else if constexpr (f * kMul / F == n) {
          // round u multiplies while round u + 1 is converted; block 0's factors are free
          // after round 0, block 1's after round 2
          convert(u < 3 ? set : set ^ 1, f, (u + 1) & 3);
          if constexpr (u == 1) set_scale(0, set ^ 1, 0, t1, f);
          if constexpr (u == 3) set_scale(1, set ^ 1, 1, t1, f);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    pin();
    la.next(g.a);
    lb.next(g.b);
    // Half t + 2 has landed.  In a unit's first two phases it has anyway (see below), and the
    // stores of the unit before may take longer.
    if (slot >= 2 || t >= 4) __builtin_amdgcn_s_waitcnt(wait_code(2 * kLoads, 15));
    __builtin_amdgcn_s_waitcnt(wait_code(63, 0));
    barrier();
  };

  int id = blockIdx.x;
  Unit unit = unit_of(id), ahead = unit;  // ahead: the unit whose halves are being loaded
  la.start(g.a, unit.m0, unit.k0, unit.kend);
  lb.start(g.b, unit.n0, unit.k0, unit.kend);
  load_group(unit, 0, 0);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    v4i qa = la.resource(g.a), qb = lb.resource(g.b);
    settle(qa, qb);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_half(i, qa, qb, t);
    la.next(g.a);
    lb.next(g.b);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  barrier();
  read_group(0);
#pragma unroll
  for (int f = 0; f < F; ++f) {
    read_block(0, f, 0, 0);
    read_block(0, f, 1, 0);
    set_scale(0, 0, 0, 0, f);
    if constexpr (kExact) {
      set_scale(1, 0, 1, 0, f);
      convert(0, f, 0);
    }
  }
  __builtin_amdgcn_s_waitcnt(wait_code(63, 0));
  barrier();  // every wave holds half 0: its buffer can be refilled

  int buf = 0;  // of the group that is being multiplied
  for (;;) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int t = 0; t < 16; ++t) acc[i][j][t] = 0.f;
    pin();
    const int next_id = id + gridDim.x;
    for (int t = 0; t < unit.halves; t += 4) {
      const bool last = t + 4 >= unit.halves;
      if (last) {  // from here on the next unit's halves are loaded
        if (next_id < units) {
          ahead = unit_of(next_id);
          la.start(g.a, ahead.m0, ahead.k0, ahead.kend);
          lb.start(g.b, ahead.n0, ahead.k0, ahead.kend);
        } else {
          la.finish();
          lb.finish();
        }
      }
      // the next group: of this unit, or the first of the next
      const bool turn = last || (t & 4);
      phase(Const<0>{}, t, t + 1, buf);
      if (turn) load_group(ahead, last ? 0 : (t + 4) >> 3, buf ^ 1);
      phase(Const<1>{}, t + 1, t + 2, buf);
      phase(Const<2>{}, t + 2, t + 3, buf);
      buf ^= turn;
      phase(Const<3>{}, t + 3, last ? 0 : t + 4, buf);
    }
    // The accumulators are read by ordinary instructions now: the last matrix instructions have
    // to retire first.  The next unit's first halves land before the stores start, so that the
    // phases that need them do not wait for the stores.
    asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 7" ::: "memory");
    pin();
    uint8_t* stage = lds + kRing + 2 * kScaleBytes + wave * kStage;
    if (g.part)
      store_tile<true, kStage>(acc, stage, unit.m0 + wm, unit.n0 + wn, g.m, g.n,
                       g.part + int64_t(unit.part) * g.m * g.n, g.n, nullptr, 0, lane);
    else
      store_tile<kExact, kStage>(acc, stage, unit.m0 + wm, unit.n0 + wn, g.m, g.n, g.out, g.ldo, g.add, g.ldadd,
                         lane);
    if (next_id >= units) break;
    id = next_id;
    unit = ahead;
  }
}

template <int TM, int TN, bool kExact>
hipError_t launch_kind(const ProductArgs& g, bool ar, bool br, int units, hipStream_t s) {
  const int most = 256 * resident(TM, TN);  // CUs times workgroups each
  const dim3 grid((unsigned)(units < most ? units : most));
  if (ar && br)
    large_kernel<TM, TN, true, true, kExact><<<grid, 256, 0, s>>>(g, units);
  else if (ar)
    large_kernel<TM, TN, true, false, kExact><<<grid, 256, 0, s>>>(g, units);
  else if (br)
    large_kernel<TM, TN, false, true, kExact><<<grid, 256, 0, s>>>(g, units);
  else
    large_kernel<TM, TN, false, false, kExact><<<grid, 256, 0, s>>>(g, units);
  return hipGetLastError();
}

}  // namespace
}  // namespace mxfp8
