// Layer norm forward and backward (mxfp8_layernorm_forward, mxfp8_layernorm_backward) on
// gfx950.
//
// forward:  mean and variance of each row in FP32: a first mean m, then the sums of d = x - m and
//           d^2 (a second pass over the row's values), which correct it: mean = m + mean(d),
//           variance = mean(d^2) - mean(d)^2, y = (d - mean(d)) rstd gamma + beta.  The rounding of
//           m, which counts where a row's mean is far above its deviation, so leaves no trace.
// backward: with xh = (x - mean) rstd and g = gamma dy,
//           dx = rstd (g - mean(g) - xh mean(g xh)), dgamma = sum dy xh, dbeta = sum dy.
// Bound by HBM: 2 and 3 passes over rows x cols values.  A row stays in registers between its
// sums and its output (at most kVec chunks of 8 for each of kThreads threads), so
// every value is read once.  Backward, a workgroup walks a group of rows, loading the next row
// while it works on this one; its threads own columns, whose sums they keep in registers and
// leave as one partial sum per group, joined in a fixed order.  Wider rows take the plain kernels
// at the end, which read rows again.
#include <hip/hip_runtime.h>

#include "layer_internal.h"
#include "values.h"

namespace mxfp8 {
namespace {

struct Args {
  int64_t rows, cols;
  float eps;
  const void* x;
  int64_t ldx;
  const float* gamma;
  const float* beta;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  float* part;  // [groups][2][cols]: dgamma, dbeta
  float* dgamma;
  float* dbeta;
  int64_t groups;
};

// Sum over the workgroup, in a fixed order; every thread gets it.
template <int kThreads>
__device__ inline float block_sum(float v, float* scratch) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (kThreads == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += scratch[w];
  return s;
}

// The same for two values at once; `scratch` alternates between calls, so one barrier is enough.
template <int kThreads>
__device__ inline float2 block_sum2(float a, float b, float2* scratch) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    a += __shfl_xor(a, d);
    b += __shfl_xor(b, d);
  }
  if constexpr (kThreads == 64) return {a, b};
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = {a, b};
  __syncthreads();
  float2 s = {0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    s.x += scratch[w].x;
    s.y += scratch[w].y;
  }
  return s;
}

// A first mean, rounded to FP32 here: without this the compiler subtracts the unrounded product from
// the values, and `off` would belong to another mean than the one it is added to.
__device__ inline float first_mean(float sum, float inv) {
  float mean = sum * inv;
  asm("" : "+v"(mean));
  return mean;
}

__device__ inline bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// 1 / sqrt(variance + eps) from the mean square of the deviations from a value that is `off` below
// the mean.  Rounding may take a variance of 0 below it; an infinity or NaN stays one.
__device__ inline float rstd_of(float square, float off, float eps) {
  const float var = finite(square) ? fmaxf(square - off * off, 0.f) : square;
  return 1.f / sqrtf(var + eps);
}

template <bool kBF16, int kThreads, int kVec>
__global__ __launch_bounds__(kThreads) void forward_row_kernel(const Args g) {
  __shared__ float scratch[kThreads / 64];
  __shared__ float2 scratch2[kThreads / 64];
  const float inv = 1.f / (float)g.cols;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    Raw<kBF16> raw[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = 8 * (int64_t)(i * kThreads + threadIdx.x);
      raw[i] = load_raw<kBF16>(g.x, c < g.cols ? r * g.ldx + c : 0, g.cols - c);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const Chunk x = values_of<kBF16>(raw[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x.v[e];
    }
    const float mean = first_mean(block_sum<kThreads>(s, scratch), inv);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t n = g.cols - 8 * (int64_t)(i * kThreads + threadIdx.x);
      const Chunk x = values_of<kBF16>(raw[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = e < n ? x.v[e] - mean : 0.f;
        s1 += d;
        s2 += d * d;
      }
    }
    const float2 t = block_sum2<kThreads>(s1, s2, scratch2);
    const float off = t.x * inv, rstd = rstd_of(t.y * inv, off, g.eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = 8 * (int64_t)(i * kThreads + threadIdx.x), n = g.cols - c;
      if (n <= 0) break;
      Chunk x = values_of<kBF16>(raw[i]), ga, be;
#pragma unroll
      for (int e = 0; e < 8; ++e) ga.v[e] = 1.f, be.v[e] = 0.f;
      if (g.gamma) ga = load8<false>(g.gamma, c, n);
      if (g.beta) be = load8<false>(g.beta, c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] = (x.v[e] - mean - off) * rstd * ga.v[e] + be.v[e];
      store8<kBF16>(g.y, r * g.ldy + c, n, x);
    }
    if (threadIdx.x == 0) {
      if (g.mean) g.mean[r] = finite(mean) ? mean + off : mean;
      if (g.rstd) g.rstd[r] = rstd;
    }
  }
}

template <bool kBF16, int kThreads, int kVec>
__global__ __launch_bounds__(kThreads) void backward_group_kernel(const Args g) {
  __shared__ float2 scratch[2][kThreads / 64];
  const float inv = 1.f / (float)g.cols;
  Raw<kBF16> x[kVec], d[kVec];
  Chunk sg[kVec], sb[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sg[i].v[e] = sb[i].v[e] = 0.f;
  auto load = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = 8 * (int64_t)(i * kThreads + threadIdx.x), n = g.cols - c;
      x[i] = load_raw<kBF16>(g.x, n > 0 ? r * g.ldx + c : 0, n);
      d[i] = load_raw<kBF16>(g.dy, n > 0 ? r * g.lddy + c : 0, n);
    }
  };
  int64_t r = blockIdx.x;
  load(r);
  float mean = g.mean[r], rstd = g.rstd[r];
  for (int turn = 0; r < g.rows; r += g.groups, turn ^= 1) {
    Raw<kBF16> xr[kVec], dr[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) xr[i] = x[i], dr[i] = d[i];
    const float m = mean, rs = rstd;
    const int64_t next = r + g.groups;
    if (next < g.rows) {
      load(next);
      mean = g.mean[next];
      rstd = g.rstd[next];
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = 8 * (int64_t)(i * kThreads + threadIdx.x), n = g.cols - c;
      if (n <= 0) break;
      const Chunk xv = values_of<kBF16>(xr[i]), dv = values_of<kBF16>(dr[i]);
      Chunk ga;
#pragma unroll
      for (int e = 0; e < 8; ++e) ga.v[e] = 1.f;
      if (g.gamma) ga = load8<false>(g.gamma, c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (xv.v[e] - m) * rs, gd = ga.v[e] * dv.v[e];
        s1 += gd;
        s2 += gd * xh;
        sg[i].v[e] += dv.v[e] * xh;
        sb[i].v[e] += dv.v[e];
      }
    }
    if (!g.dx) continue;
    const float2 t = block_sum2<kThreads>(s1, s2, scratch[turn]);
    const float m1 = t.x * inv, m2 = t.y * inv;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = 8 * (int64_t)(i * kThreads + threadIdx.x), n = g.cols - c;
      if (n <= 0) break;
      const Chunk xv = values_of<kBF16>(xr[i]);
      Chunk dv = values_of<kBF16>(dr[i]), ga;
#pragma unroll
      for (int e = 0; e < 8; ++e) ga.v[e] = 1.f;
      if (g.gamma) ga = load8<false>(g.gamma, c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dv.v[e] = rs * (ga.v[e] * dv.v[e] - m1 - (xv.v[e] - m) * rs * m2);
      store8<kBF16>(g.dx, r * g.lddx + c, n, dv);
    }
  }
  if (!g.part) return;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t c = 8 * (int64_t)(i * kThreads + threadIdx.x), n = g.cols - c;
    if (n <= 0) break;
    store8<false, false>(g.part, (2 * blockIdx.x) * g.cols + c, n, sg[i]);
    store8<false, false>(g.part, (2 * blockIdx.x + 1) * g.cols + c, n, sb[i]);
  }
}

// ---- rows too wide for the registers

// A compensated sum: the rounding of each addition is carried into the next, so a thread's sum is as
// exact over millions of columns as over a few.  Infinities and NaN sum as they do in plain additions.
struct Sum {
  float s = 0.f, c = 0.f;
  __device__ inline void add(float v) {
    const float y = v - c, t = s + y;
    c = finite(t) ? (t - s) - y : 0.f;
    s = t;
  }
  // 8 values, joined in a tree first
  __device__ inline void add(const float (&v)[8]) {
    add(((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7])));
  }
};

template <bool kBF16>
__global__ __launch_bounds__(256) void forward_kernel(const Args g) {
  __shared__ float scratch[4];
  __shared__ float2 scratch2[4];
  const float inv = 1.f / (float)g.cols;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const int64_t base = r * g.ldx;
    Sum s;
    for (int64_t c = 8 * threadIdx.x; c < g.cols; c += 2048)
      s.add(load8<kBF16>(g.x, base + c, g.cols - c).v);
    const float mean = first_mean(block_sum<256>(s.s, scratch), inv);
    Sum s1, s2;
    for (int64_t c = 8 * threadIdx.x; c < g.cols; c += 2048) {
      const Chunk x = load8<kBF16>(g.x, base + c, g.cols - c);
      float d[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = c + i < g.cols ? x.v[i] - mean : 0.f;
        q[i] = d[i] * d[i];
      }
      s1.add(d);
      s2.add(q);
    }
    const float2 t = block_sum2<256>(s1.s, s2.s, scratch2);
    const float off = t.x * inv, rstd = rstd_of(t.y * inv, off, g.eps);
    for (int64_t c = 8 * threadIdx.x; c < g.cols; c += 2048) {
      const int64_t n = g.cols - c;
      Chunk x = load8<kBF16>(g.x, base + c, n), ga, be;
#pragma unroll
      for (int i = 0; i < 8; ++i) ga.v[i] = 1.f, be.v[i] = 0.f;
      if (g.gamma) ga = load8<false>(g.gamma, c, n);
      if (g.beta) be = load8<false>(g.beta, c, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) x.v[i] = (x.v[i] - mean - off) * rstd * ga.v[i] + be.v[i];
      store8<kBF16>(g.y, r * g.ldy + c, n, x);
    }
    if (threadIdx.x == 0) {
      if (g.mean) g.mean[r] = finite(mean) ? mean + off : mean;
      if (g.rstd) g.rstd[r] = rstd;
    }
  }
}

template <bool kBF16>
__global__ __launch_bounds__(256) void backward_rows_kernel(const Args g) {
  __shared__ float scratch[4];
  const float inv = 1.f / (float)g.cols;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const float mean = g.mean[r], rstd = g.rstd[r];
    Sum s1, s2;
    for (int64_t c = 8 * threadIdx.x; c < g.cols; c += 2048) {
      const int64_t n = g.cols - c;
      const Chunk x = load8<kBF16>(g.x, r * g.ldx + c, n), d = load8<kBF16>(g.dy, r * g.lddy + c, n);
      Chunk ga;
#pragma unroll
      for (int i = 0; i < 8; ++i) ga.v[i] = 1.f;
      if (g.gamma) ga = load8<false>(g.gamma, c, n);
      float gd[8], gx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gd[i] = ga.v[i] * d.v[i];
        gx[i] = gd[i] * ((x.v[i] - mean) * rstd);
      }
      s1.add(gd);
      s2.add(gx);
    }
    const float m1 = block_sum<256>(s1.s, scratch) * inv;
    const float m2 = block_sum<256>(s2.s, scratch) * inv;
    for (int64_t c = 8 * threadIdx.x; c < g.cols; c += 2048) {
      const int64_t n = g.cols - c;
      const Chunk x = load8<kBF16>(g.x, r * g.ldx + c, n);
      Chunk d = load8<kBF16>(g.dy, r * g.lddy + c, n), ga;
#pragma unroll
      for (int i = 0; i < 8; ++i) ga.v[i] = 1.f;
      if (g.gamma) ga = load8<false>(g.gamma, c, n);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d.v[i] = rstd * (ga.v[i] * d.v[i] - m1 - (x.v[i] - mean) * rstd * m2);
      store8<kBF16>(g.dx, r * g.lddx + c, n, d);
    }
  }
}

// Partial dgamma and dbeta of the rows of one group (rows group, group + groups, ...).
template <bool kBF16>
__global__ __launch_bounds__(256) void backward_cols_kernel(const Args g) {
  const int64_t c = 8 * (int64_t(blockIdx.x) * 256 + threadIdx.x);
  if (c >= g.cols) return;
  const int64_t n = g.cols - c;
  Chunk sg, sb;
#pragma unroll
  for (int i = 0; i < 8; ++i) sg.v[i] = sb.v[i] = 0.f;
  for (int64_t r = blockIdx.y; r < g.rows; r += g.groups) {
    const float mean = g.mean[r], rstd = g.rstd[r];
    const Chunk x = load8<kBF16>(g.x, r * g.ldx + c, n), d = load8<kBF16>(g.dy, r * g.lddy + c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sg.v[i] += d.v[i] * ((x.v[i] - mean) * rstd);
      sb.v[i] += d.v[i];
    }
  }
  store8<false, false>(g.part, (2 * blockIdx.y) * g.cols + c, n, sg);
  store8<false, false>(g.part, (2 * blockIdx.y + 1) * g.cols + c, n, sb);
}

// Joins the groups' partial sums: 32 columns a workgroup, 8 slices of the groups each summed in
// order, then the slices in order.  blockIdx.y: dgamma or dbeta.
__global__ __launch_bounds__(256) void join_kernel(const Args g) {
  __shared__ float slice[8][32];
  const int which = blockIdx.y, k0 = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31);
  float s = 0.f;
  if (c < g.cols) {
#pragma unroll 8
    for (int64_t k = k0; k < g.groups; k += 8) s += g.part[(2 * k + which) * g.cols + c];
  }
  slice[k0][threadIdx.x & 31] = s;
  __syncthreads();
  if (k0 != 0 || c >= g.cols) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += slice[k][threadIdx.x];
  float* out = which ? g.dbeta : g.dgamma;
  if (out) out[c] = s;
}

Args args_of(const mxfp8_layernorm& p) {
  Args g{};
  g.rows = p.rows;
  g.cols = p.cols;
  g.eps = p.eps;
  g.x = p.x.ptr;
  g.ldx = p.x.ld;
  g.gamma = p.gamma;
  g.beta = p.beta;
  g.y = p.y.ptr;
  g.ldy = p.y.ld;
  g.mean = p.mean;
  g.rstd = p.rstd;
  g.dy = p.dy.ptr;
  g.lddy = p.dy.ld;
  g.dx = p.dx.ptr;
  g.lddx = p.dx.ld;
  g.part = static_cast<float*>(p.workspace);
  g.dgamma = p.dgamma;
  g.dbeta = p.dbeta;
  g.groups = layernorm_groups(p.rows, p.cols);
  return g;
}

// Workgroups of a kernel that takes a row each, in turn: a launch holds fewer than 2^32 threads.
unsigned row_grid(const Args& g) { return (unsigned)(g.rows < (1 << 20) ? g.rows : 1 << 20); }

template <bool kBF16, int kThreads, int kVec>
void run_rows(const Args& g, bool backward, hipStream_t s) {
  if (backward)
    backward_group_kernel<kBF16, kThreads, kVec><<<dim3((unsigned)g.groups), kThreads, 0, s>>>(g);
  else
    forward_row_kernel<kBF16, kThreads, kVec><<<dim3(row_grid(g)), kThreads, 0, s>>>(g);
}

// The kernels that hold a row in registers: the fewest threads that do so with up to 4 chunks
// each; one wave needs no barrier.
template <bool kBF16, int kThreads>
void run_width(const Args& g, bool backward, hipStream_t s) {
  const int64_t vec = (g.cols + 8 * kThreads - 1) / (8 * kThreads);
  if (vec <= 1)
    run_rows<kBF16, kThreads, 1>(g, backward, s);
  else if (vec == 2)
    run_rows<kBF16, kThreads, 2>(g, backward, s);
  else if (vec == 3)
    run_rows<kBF16, kThreads, 3>(g, backward, s);
  else
    run_rows<kBF16, kThreads, 4>(g, backward, s);
}

template <bool kBF16>
void run(const Args& g, bool backward, hipStream_t s) {
  if (g.cols <= 2048)
    run_width<kBF16, 64>(g, backward, s);
  else if (g.cols <= 8192)
    run_width<kBF16, 256>(g, backward, s);
  else
    run_width<kBF16, 512>(g, backward, s);
}

}  // namespace

hipError_t launch_layernorm_forward(const mxfp8_layernorm& p, hipStream_t s) {
  const Args g = args_of(p);
  const dim3 grid(row_grid(g));
  if (layernorm_in_registers(p.cols)) {
    if (p.dtype == MXFP8_BF16)
      run<true>(g, false, s);
    else
      run<false>(g, false, s);
  } else if (p.dtype == MXFP8_BF16) {
    forward_kernel<true><<<grid, 256, 0, s>>>(g);
  } else {
    forward_kernel<false><<<grid, 256, 0, s>>>(g);
  }
  return hipGetLastError();
}

hipError_t launch_layernorm_backward(const mxfp8_layernorm& p, hipStream_t s) {
  Args g = args_of(p);
  const bool bf16 = p.dtype == MXFP8_BF16, sums = p.dgamma || p.dbeta;
  if (!sums) g.part = nullptr;
  if (p.rows > 0) {
    if (layernorm_in_registers(p.cols)) {
      if (bf16)
        run<true>(g, true, s);
      else
        run<false>(g, true, s);
    } else {
      if (sums) {  // first: dx may overwrite dy
        const dim3 grid((unsigned)((p.cols + 2047) / 2048), (unsigned)g.groups);
        if (bf16)
          backward_cols_kernel<true><<<grid, 256, 0, s>>>(g);
        else
          backward_cols_kernel<false><<<grid, 256, 0, s>>>(g);
      }
      if (p.dx.ptr) {
        if (bf16)
          backward_rows_kernel<true><<<dim3(row_grid(g)), 256, 0, s>>>(g);
        else
          backward_rows_kernel<false><<<dim3(row_grid(g)), 256, 0, s>>>(g);
      }
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !sums) return e;
  }
  join_kernel<<<dim3((unsigned)((p.cols + 31) / 32), 2), 256, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace mxfp8
