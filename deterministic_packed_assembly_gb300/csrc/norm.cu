// Layer norm of packed positions, and its gradients.
//
//   m = mean of x, r = 1 / sqrt(mean of (x - m)^2 + eps), xh = (x - m) r, y = xh w + b
//   g = dy w,  dx = r (g - mean of g - xh mean of (g xh))
//   dw = sum of dy xh and db = sum of dy over the positions
//
// Memory bounds both passes: a row is read once and kept in registers, as it lies in
// memory, by as few warps as hold it; the variance is taken from the kept values less
// their mean, so that a mean far from 0 costs no digits.  A lane's columns are the same in
// every row, eight at a time (rows.cuh).  What is next to bound it is instructions: they go
// by pairs (elem.cuh), and values are widened again for each use.
//
// Backward a group of warps walks rows, the next one's loads under way, and keeps the sums of
// its columns' dw and db in registers; blocks write them out once, and the last kernel adds
// the blocks' rows in order.  Rows of more columns than that (kKept) are read twice by the kernel of dx, the
// second time from the caches, and once more by that of dw and db.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "train.h"

namespace nsk {
namespace {

constexpr uint32_t kSMs = 152;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kForwardWarps = 8;      // of a block forward, and at most of a row
constexpr int kMostWarps = 16;        // of a row backward
constexpr uint32_t kKept = 8192;      // columns of the backward pass in registers
constexpr int kWideThreads = 512;     // of a row that is not kept
constexpr int kColumnWarps = 8;       // of 256 columns' sums

struct NormParams {
  const void *x, *dy, *weight, *bias;
  int64_t x_row, dy_row;
  const int32_t *doc;
  void *y;               // or dx
  float *mean, *rstd;
  float eps;
  uint32_t N, D;
  uint32_t lanes, warps;  // of a row: lanes of one warp, or warps
  float *partial;         // [blocks][2][D]
  void *dweight, *dbias;
  uint32_t blocks;
};

// ---- sums over a row's lanes ------------------------------------------------------------
__device__ __forceinline__ float lanes_sum(float v, uint32_t lanes) {
  for (uint32_t o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// Barrier of a group of warps.
__device__ __forceinline__ void group_sync(uint32_t group, uint32_t warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}

// Eight columns of a weight vector, `otherwise` where there is none.
template <class W, int V>
__device__ __forceinline__ void load_vector(const void *p, uint32_t c, uint32_t step, uint32_t D,
                                            float otherwise, Ch<2> (&v)[kOct / 2]) {
  if (p) {
    Oct<W, V> x;
    clear(x);
    load_oct(x, static_cast<const W *>(p), c, step, D);
    widen(x, v);
  } else {
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) v[j] = splat<2>(otherwise);
  }
}

// Whether column j of a lane's eight is in the row.
template <int V>
__device__ __forceinline__ bool inside(uint32_t c, uint32_t step, uint32_t D, int j) {
  return c + j / V * step + j % V < D;
}

// ---- forward --------------------------------------------------------------------------
// Rows of `lanes` lanes of a warp, or of `warps` warps; a lane has NC spans of each.
template <class E, class W, int NC, int V>
__global__ void __launch_bounds__(32 * kForwardWarps, 3) norm_forward_kernel(const NormParams p) {
  __shared__ float sums[2][kForwardWarps];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t group = warp / p.warps, part = warp % p.warps;
  const uint32_t groups = blockDim.x / 32 / p.warps, per = 32 / p.lanes;
  const uint64_t n = ((uint64_t)blockIdx.x * groups + group) * per + lane / p.lanes;
  const bool real = n < p.N, there = real && !(p.doc && p.doc[n] < 0);
  const uint32_t span = p.lanes * kOct, step = p.lanes * V;
  const uint32_t first = part * NC * span + lane % p.lanes * V;
  const E *x = static_cast<const E *>(p.x) + (int64_t)(real ? n : 0) * p.x_row;
  E *y = static_cast<E *>(p.y) + (int64_t)(real ? n : 0) * p.D;
  const float share = 1.0f / (float)p.D;
  Oct<E, V> v[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    clear(v[i]);
    if (there) load_oct(v[i], x, first + i * span, step, p.D);
  }
  Ch<2> two = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    Ch<2> f[kOct / 2];
    widen(v[i], f);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) two = two + f[j];
  }
  float sum = lanes_sum(two.v[0] + two.v[1], p.lanes);
  if (p.warps > 1) {
    if (lane == 0) sums[0][warp] = sum;
    group_sync(group, p.warps);
    sum = 0.0f;
    for (uint32_t w = 0; w < p.warps; ++w) sum += sums[0][group * p.warps + w];
  }
  const float mean = sum * share;
  const Ch<2> minus = splat<2>(-mean);
  two = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t c = first + i * span;
    Ch<2> f[kOct / 2];
    forget(v[i]);
    widen(v[i], f);
    // a span that ends beyond the row: what is not there has no part
    const bool all = first - lane % p.lanes * V + (i + 1) * span <= p.D;
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      Ch<2> d = f[j] + minus;
      if (!all) {
        if (!inside<V>(c, step, p.D, 2 * j)) d.v[0] = 0.0f;
        if (!inside<V>(c, step, p.D, 2 * j + 1)) d.v[1] = 0.0f;
      }
      two = fma(d, d, two);
    }
  }
  float square = lanes_sum(two.v[0] + two.v[1], p.lanes);
  if (p.warps > 1) {
    if (lane == 0) sums[1][warp] = square;
    group_sync(group, p.warps);
    square = 0.0f;
    for (uint32_t w = 0; w < p.warps; ++w) square += sums[1][group * p.warps + w];
  }
  const float rstd = __frsqrt_rn(fmaf(square, share, p.eps));
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t c = first + i * span;
    if (c >= p.D) break;
    Ch<2> f[kOct / 2], w[kOct / 2], b[kOct / 2];
    load_vector<W, V>(p.weight, c, step, p.D, 1.0f, w);
    load_vector<W, V>(p.bias, c, step, p.D, 0.0f, b);
    forget(v[i]);
    widen(v[i], f);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      f[j] = fma((f[j] + minus) * splat<2>(rstd), w[j], b[j]);
      if (!there) f[j] = {0.0f, 0.0f};
    }
    if (real) store_oct(y, c, step, p.D, narrow<E, V>(f));
  }
  if (real && part == 0 && lane % p.lanes == 0) {
    if (p.mean) p.mean[n] = there ? mean : 0.0f;
    if (p.rstd) p.rstd[n] = there ? rstd : 0.0f;
  }
}

// The sum of v over a block, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float *sums) {
  v = lanes_sum(v, 32);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kWideThreads / 32; ++w) v += sums[w];
  return v;
}

// A block a row of any width, read three times.
template <class E, class W, int V>
__global__ void __launch_bounds__(kWideThreads) norm_forward_wide_kernel(const NormParams p) {
  __shared__ float sums[kWideThreads / 32];
  const uint32_t n = blockIdx.x, lane = threadIdx.x % 32, D = p.D;
  const bool there = !(p.doc && p.doc[n] < 0);
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  E *y = static_cast<E *>(p.y) + (int64_t)n * D;
  constexpr uint32_t kStep = 32 * V, kAll = kWideThreads * kOct;
  const uint32_t c0 = threadIdx.x / 32 * 32 * kOct + lane * V;
  const float share = 1.0f / (float)D;
  float mean = 0.0f, rstd = 0.0f;
  Ch<2> f[kOct / 2], two = {0.0f, 0.0f};
  Oct<E, V> v;
  clear(v);
  if (there) {
    for (uint32_t c = c0; c < D; c += kAll) {
      clear(v);
      load_oct(v, x, c, kStep, D);
      widen(v, f);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) two = two + f[j];
    }
    mean = block_sum(two.v[0] + two.v[1], sums) * share;
    two = {0.0f, 0.0f};
    for (uint32_t c = c0; c < D; c += kAll) {
      load_oct(v, x, c, kStep, D);
      widen(v, f);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) {
        Ch<2> d = f[j] + splat<2>(-mean);
        if (!inside<V>(c, kStep, D, 2 * j)) d.v[0] = 0.0f;
        if (!inside<V>(c, kStep, D, 2 * j + 1)) d.v[1] = 0.0f;
        two = fma(d, d, two);
      }
    }
    rstd = __frsqrt_rn(fmaf(block_sum(two.v[0] + two.v[1], sums), share, p.eps));
  }
  for (uint32_t c = c0; c < D; c += kAll) {
    Ch<2> w[kOct / 2], b[kOct / 2];
    load_vector<W, V>(p.weight, c, kStep, D, 1.0f, w);
    load_vector<W, V>(p.bias, c, kStep, D, 0.0f, b);
    if (there) load_oct(v, x, c, kStep, D);
    widen(v, f);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      f[j] = fma((f[j] + splat<2>(-mean)) * splat<2>(rstd), w[j], b[j]);
      if (!there) f[j] = {0.0f, 0.0f};
    }
    store_oct(y, c, kStep, D, narrow<E, V>(f));
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[n] = mean;
    if (p.rstd) p.rstd[n] = rstd;
  }
}

// ---- backward -----------------------------------------------------------------------
// Groups of `warps` warps (or of `lanes` lanes) walk rows; a lane has NC spans of each.
constexpr int kBackWarps = 10;   // of a block of rows of up to as many warps
constexpr uint32_t kNarrow = 32 * kOct * kMostWarps;  // columns up to which NC is 1

// Blocks of an SM: as many as have registers for the sums, a row and the next one.
template <class E, int V, int NC, int kThreads>
constexpr int kBackBlocks = NC > 1 ? 1
                            : Oct<E, V>::kPieces * Oct<E, V>::kWords == 4
                                ? (kThreads > 320 ? 2 : 3)
                                : (kThreads > 320 ? 1 : 2);

// A row's values as they lie, its statistics, and whether it is one.
template <class E, int NC, int V>
struct NormRow {
  Oct<E, V> x[NC], g[NC];
  float mean, rstd;
  bool real, there;
};
template <class E, int NC, int V>
__device__ __forceinline__ void load_row(NormRow<E, NC, V> &r, const NormParams &p, uint64_t n,
                                         uint32_t first, uint32_t span, uint32_t step) {
  r.real = n < p.N;
  r.there = r.real && !(p.doc && p.doc[n] < 0);
  r.mean = r.rstd = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) clear(r.x[i]), clear(r.g[i]);
  if (!r.there) return;
  r.mean = p.mean[n], r.rstd = p.rstd[n];
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  const E *dy = static_cast<const E *>(p.dy) + (int64_t)n * p.dy_row;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    load_oct(r.x[i], x, first + i * span, step, p.D);
    load_oct(r.g[i], dy, first + i * span, step, p.D);
  }
}

template <class E, class W, int NC, int V, int kThreads>
__global__ void __launch_bounds__(kThreads, (kBackBlocks<E, V, NC, kThreads>))
    norm_backward_kernel(const NormParams p) {
  __shared__ float2 sums[2][kThreads / 32];
  extern __shared__ float joined[];  // [2][columns]: the groups' sums
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t group = warp / p.warps, part = warp % p.warps;
  const uint32_t groups = blockDim.x / 32 / p.warps, per = 32 / p.lanes;
  const uint32_t span = p.lanes * kOct, step = p.lanes * V;
  const uint32_t first = part * NC * span + lane % p.lanes * V;
  const float share = 1.0f / (float)p.D;
  Ch<2> w[NC][kOct / 2], dw[NC][kOct / 2], db[NC][kOct / 2];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) dw[i][j] = db[i][j] = {0.0f, 0.0f};
    load_vector<W, V>(p.weight, first + i * span, step, p.D, 1.0f, w[i]);
  }
  const uint64_t every = (uint64_t)gridDim.x * groups * per;
  uint32_t turn = 0;
  // a group's lanes stay together: rows from the first lane's on
  uint64_t n0 = ((uint64_t)blockIdx.x * groups + group) * per;
  NormRow<E, NC, V> row;
  load_row(row, p, n0 + lane / p.lanes, first, span, step);
  for (; n0 < p.N; n0 += every) {
    NormRow<E, NC, V> next;
    load_row(next, p, n0 + every + lane / p.lanes, first, span, step);
    const Ch<2> minus = splat<2>(-row.mean), scale = splat<2>(row.rstd);
    Ch<2> s1 = {0.0f, 0.0f}, s2 = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      Ch<2> f[kOct / 2], g[kOct / 2];
      widen(row.x[i], f);
      widen(row.g[i], g);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) {
        const Ch<2> xh = (f[j] + minus) * scale, gw = g[j] * w[i][j];
        s1 = s1 + gw;
        s2 = fma(gw, xh, s2);
        dw[i][j] = fma(g[j], xh, dw[i][j]);
        db[i][j] = db[i][j] + g[j];
      }
    }
    float a = lanes_sum(s1.v[0] + s1.v[1], p.lanes), b = lanes_sum(s2.v[0] + s2.v[1], p.lanes);
    if (p.warps > 1) {  // two buffers: one barrier a row
      if (lane == 0) sums[turn][warp] = make_float2(a, b);
      group_sync(group, p.warps);
      a = b = 0.0f;
      for (uint32_t k = 0; k < p.warps; ++k) {
        const float2 v = sums[turn][group * p.warps + k];
        a += v.x, b += v.y;
      }
      turn ^= 1;
    }
    const Ch<2> m1 = splat<2>(-a * share), m2 = splat<2>(-b * share);
    if (row.real) {
      E *dx = static_cast<E *>(p.y) + (int64_t)(n0 + lane / p.lanes) * p.D;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        Ch<2> f[kOct / 2], g[kOct / 2];
        forget(row.x[i]), forget(row.g[i]);
        widen(row.x[i], f);
        widen(row.g[i], g);
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) {
          const Ch<2> xh = (f[j] + minus) * scale;
          f[j] = scale * fma(xh, m2, fma(g[j], w[i][j], m1));
          if (!row.there) f[j] = {0.0f, 0.0f};
        }
        store_oct(dx, first + i * span, step, p.D, narrow<E, V>(f));
      }
    }
    row = next;
  }
  if (!p.partial) return;
  // lanes that share columns, then groups that do, in order
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j)
      for (uint32_t o = p.lanes; o < 32; o <<= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          dw[i][j].v[h] += __shfl_xor_sync(kFull, dw[i][j].v[h], o);
          db[i][j].v[h] += __shfl_xor_sync(kFull, db[i][j].v[h], o);
        }
  const uint32_t columns = p.warps * NC * span;
  for (uint32_t g = 0; g < groups; ++g) {
    if (g == group && lane < p.lanes) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < kOct; ++j) {
          float *a = joined + first + i * span + j / V * step + j % V, *b = a + columns;
          const float u = dw[i][j / 2].v[j & 1], v = db[i][j / 2].v[j & 1];
          *a = g ? *a + u : u;
          *b = g ? *b + v : v;
        }
    }
    __syncthreads();
  }
  float *to = p.partial + (uint64_t)blockIdx.x * 2 * p.D;
  for (uint32_t c = threadIdx.x; c < p.D; c += blockDim.x) {
    to[c] = joined[c];
    to[p.D + c] = joined[columns + c];
  }
}

// A block a row of any width, read twice.
template <class E, class W, int V>
__global__ void __launch_bounds__(kWideThreads) norm_backward_wide_kernel(const NormParams p) {
  __shared__ float sums[kWideThreads / 32];
  const uint32_t n = blockIdx.x, lane = threadIdx.x % 32, D = p.D;
  const bool there = !(p.doc && p.doc[n] < 0);
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  const E *dy = static_cast<const E *>(p.dy) + (int64_t)n * p.dy_row;
  E *dx = static_cast<E *>(p.y) + (int64_t)n * D;
  constexpr uint32_t kStep = 32 * V, kAll = kWideThreads * kOct;
  const uint32_t c0 = threadIdx.x / 32 * 32 * kOct + lane * V;
  Ch<2> s1 = {0.0f, 0.0f}, s2 = s1, minus = s1, scale = s1, m1 = s1, m2 = s1;
  Ch<2> f[kOct / 2], g[kOct / 2], w[kOct / 2];
  Oct<E, V> xv, gv;
  clear(xv), clear(gv);
  if (there) {
    minus = splat<2>(-p.mean[n]), scale = splat<2>(p.rstd[n]);
    for (uint32_t c = c0; c < D; c += kAll) {
      clear(gv);
      load_oct(xv, x, c, kStep, D);
      load_oct(gv, dy, c, kStep, D);
      load_vector<W, V>(p.weight, c, kStep, D, 1.0f, w);
      widen(xv, f);
      widen(gv, g);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) {
        const Ch<2> gw = g[j] * w[j];
        s1 = s1 + gw;
        s2 = fma(gw, (f[j] + minus) * scale, s2);
      }
    }
    m1 = splat<2>(-block_sum(s1.v[0] + s1.v[1], sums) / (float)D);
    m2 = splat<2>(-block_sum(s2.v[0] + s2.v[1], sums) / (float)D);
  }
  for (uint32_t c = c0; c < D; c += kAll) {
    if (there) {
      load_oct(xv, x, c, kStep, D);
      load_oct(gv, dy, c, kStep, D);
    }
    load_vector<W, V>(p.weight, c, kStep, D, 1.0f, w);
    widen(xv, f);
    widen(gv, g);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      f[j] = scale * fma((f[j] + minus) * scale, m2, fma(g[j], w[j], m1));
      if (!there) f[j] = {0.0f, 0.0f};
    }
    store_oct(dx, c, kStep, D, narrow<E, V>(f));
  }
}

// Rows y, y + blocks, ... of 256 columns.
template <class E, int V>
__global__ void __launch_bounds__(32 * kColumnWarps) norm_columns_kernel(const NormParams p) {
  __shared__ float sums[kColumnWarps][2][32 * kOct];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t c = blockIdx.x * 32 * kOct + lane * V;
  Ch<2> dw[kOct / 2], db[kOct / 2];
#pragma unroll
  for (int j = 0; j < kOct / 2; ++j) dw[j] = db[j] = {0.0f, 0.0f};
#pragma unroll 2
  for (uint64_t n = (uint64_t)blockIdx.y * kColumnWarps + warp; n < p.N;
       n += (uint64_t)gridDim.y * kColumnWarps) {
    if (p.doc && p.doc[n] < 0) continue;
    Oct<E, V> xv, gv;
    clear(xv), clear(gv);
    load_oct(xv, static_cast<const E *>(p.x) + (int64_t)n * p.x_row, c, 32 * V, p.D);
    load_oct(gv, static_cast<const E *>(p.dy) + (int64_t)n * p.dy_row, c, 32 * V, p.D);
    const Ch<2> minus = splat<2>(-p.mean[n]), scale = splat<2>(p.rstd[n]);
    Ch<2> f[kOct / 2], g[kOct / 2];
    widen(xv, f);
    widen(gv, g);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      dw[j] = fma(g[j], (f[j] + minus) * scale, dw[j]);
      db[j] = db[j] + g[j];
    }
  }
#pragma unroll
  for (int j = 0; j < kOct; ++j) {
    sums[warp][0][j / V * 32 * V + lane * V + j % V] = dw[j / 2].v[j & 1];
    sums[warp][1][j / V * 32 * V + lane * V + j % V] = db[j / 2].v[j & 1];
  }
  __syncthreads();
  const uint64_t col = (uint64_t)blockIdx.x * 32 * kOct + threadIdx.x;
  if (col < p.D) {
    float a = 0.0f, b = 0.0f;
    for (int k = 0; k < kColumnWarps; ++k) a += sums[k][0][threadIdx.x], b += sums[k][1][threadIdx.x];
    float *to = p.partial + (uint64_t)blockIdx.y * 2 * p.D;
    to[col] = a, to[p.D + col] = b;
  }
}

// The blocks' rows, added in order: 32 columns a block, eight runs of rows.
template <class W>
__global__ void __launch_bounds__(256) norm_total_kernel(const NormParams p) {
  pdl_wait();
  __shared__ float sums[8][33];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
  const uint32_t run = (p.blocks + 7) / 8, a = min(p.blocks, warp * run), b = min(p.blocks, a + run);
  for (int which = 0; which < 2; ++which) {
    W *to = static_cast<W *>(which ? p.dbias : p.dweight);
    if (!to) continue;
    float sum = 0.0f;
    if (c < p.D) {
#pragma unroll 8
      for (uint32_t i = a; i < b; ++i) sum += p.partial[((uint64_t)i * 2 + which) * p.D + c];
    }
    __syncthreads();
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < p.D) {
      for (int k = 1; k < 8; ++k) sum += sums[k][lane];
      to[c] = from_f32<W>(sum);
    }
  }
}

// ---- launches -----------------------------------------------------------------------
template <class E, class W, int NC, int V>
cudaError_t launch_forward(const NormParams &p, uint32_t threads, uint32_t rows, cudaStream_t st) {
  norm_forward_kernel<E, W, NC, V>
      <<<(uint32_t)(((uint64_t)p.N + rows - 1) / rows), threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <class E, class W, int V>
cudaError_t forward_of(NormParams &p, cudaStream_t st) {
  // a lane keeps up to 40 registers of a row
  constexpr uint32_t kMost = 40 / (Oct<E, V>::kPieces * Oct<E, V>::kWords);
  p.lanes = lanes_for(p.D);
  const uint64_t spans = spans_for(p.D, p.lanes);
  ++launch_counter();
  if (spans > kMost * kForwardWarps) {
    norm_forward_wide_kernel<E, W, V><<<p.N, kWideThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  p.warps = (uint32_t)((spans + kMost - 1) / kMost);
  const uint32_t nc = (uint32_t)((spans + p.warps - 1) / p.warps);
  const uint32_t groups = kForwardWarps / p.warps;
  const uint32_t threads = groups * p.warps * 32, rows = groups * (32 / p.lanes);
  switch (nc) {
    case 1: return launch_forward<E, W, 1, V>(p, threads, rows, st);
    case 2: return launch_forward<E, W, 2, V>(p, threads, rows, st);
    case 3: return launch_forward<E, W, 3, V>(p, threads, rows, st);
    case 4: return launch_forward<E, W, 4, V>(p, threads, rows, st);
    case 5: return launch_forward<E, W, 5, V>(p, threads, rows, st);
    default:
      if constexpr (kMost > 5) {
        if (nc <= 6) return launch_forward<E, W, 6, V>(p, threads, rows, st);
        if (nc <= 8) return launch_forward<E, W, 8, V>(p, threads, rows, st);
        return launch_forward<E, W, 10, V>(p, threads, rows, st);
      }
      return cudaErrorInvalidValue;
  }
}

// The backward pass's grid, by the sizes alone: the workspace follows from it.
struct Back {
  uint32_t lanes, warps, groups, nc, blocks;  // of the kept form
  uint32_t across;                            // blocks across rows of the other form's sums
};
Back back_of(uint32_t N, uint32_t D) {
  Back b = {};
  b.lanes = lanes_for(D);
  const uint32_t spans = (uint32_t)spans_for(D, b.lanes);
  if (D > kKept) {
    // blocks of 256 columns: enough to fill the SMs, each with rows for its warps
    const uint64_t most = ((uint64_t)N + 4 * kColumnWarps - 1) / (4 * kColumnWarps);
    b.across = (uint32_t)std::min<uint64_t>(most, (8 * kSMs + spans - 1) / spans);
    b.blocks = b.across;
    return b;
  }
  b.nc = D > kNarrow ? 2 : 1;
  b.warps = (spans + b.nc - 1) / b.nc;
  b.groups = std::max<uint32_t>(1, kBackWarps / b.warps);
  const uint64_t rows = (uint64_t)b.groups * (32 / b.lanes);
  b.blocks = (uint32_t)std::min<uint64_t>(((uint64_t)N + rows - 1) / rows, 3 * kSMs);
  return b;
}

template <class E, class W, int NC, int V, int kThreads>
cudaError_t launch_backward(NormParams &p, const Back &b, cudaStream_t st) {
  const uint32_t threads = b.groups * b.warps * 32;
  const size_t shared = 2 * sizeof(float) * b.warps * NC * b.lanes * kOct;
  auto *k = norm_backward_kernel<E, W, NC, V, kThreads>;
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(k));
  if (e != cudaSuccess) return e;
  p.blocks = std::min<uint32_t>(b.blocks, kBackBlocks<E, V, NC, kThreads> * kSMs);
  ++launch_counter();
  k<<<p.blocks, threads, shared, st>>>(p);
  return cudaGetLastError();
}

template <class E, class W, int V>
cudaError_t backward_of(NormParams &p, cudaStream_t st) {
  const Back b = back_of(p.N, p.D);
  p.lanes = b.lanes, p.warps = b.warps, p.blocks = b.blocks;
  cudaError_t e = cudaSuccess;
  if (p.N && p.D > kKept) {
    ++launch_counter();
    norm_backward_wide_kernel<E, W, V><<<p.N, kWideThreads, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.partial) return e;
    ++launch_counter();
    norm_columns_kernel<E, V>
        <<<dim3((p.D + 32 * kOct - 1) / (32 * kOct), b.across), 32 * kColumnWarps, 0, st>>>(p);
    e = cudaGetLastError();
  } else if (p.N) {
    constexpr int kMost = 32 * kMostWarps, kFew = 32 * kBackWarps;
    e = b.nc == 2              ? launch_backward<E, W, 2, V, kMost>(p, b, st)
        : b.warps > kBackWarps ? launch_backward<E, W, 1, V, kMost>(p, b, st)
                               : launch_backward<E, W, 1, V, kFew>(p, b, st);
  }
  if (e != cudaSuccess || (!p.dweight && !p.dbias)) return e;
  ++launch_counter();
  pdl_launch(norm_total_kernel<W>, dim3((p.D + 31) / 32), dim3(256), 0, st, p);
  return cudaGetLastError();
}

NormParams params_of(const ns_norm_inputs &in) {
  NormParams p = {};
  p.x = in.x, p.x_row = in.x_row, p.weight = in.weight, p.bias = in.bias, p.doc = in.doc;
  p.N = in.N, p.D = in.D, p.eps = in.eps;
  return p;
}

// By the types of the rows and of the weights, which are floats or as the rows, and the
// pieces that all of them can be moved by.
template <class F>
cudaError_t by_types(const ns_norm_inputs &in, int piece, F &&call) {
  const auto with = [&](auto e, auto w) {
    if (piece == 8) return call(e, w, std::integral_constant<int, 8>{});
    if (piece == 2) return call(e, w, std::integral_constant<int, 2>{});
    return call(e, w, std::integral_constant<int, 1>{});
  };
  if (in.dtype == NS_F32) return with(float{}, float{});
  if (in.dtype == NS_BF16)
    return in.weight_dtype == NS_F32 ? with(__nv_bfloat16{}, float{})
                                     : with(__nv_bfloat16{}, __nv_bfloat16{});
  return in.weight_dtype == NS_F32 ? with(__half{}, float{}) : with(__half{}, __half{});
}
int piece_of_inputs(const ns_norm_inputs &in, const void *y) {
  const uint64_t es = in.dtype == NS_F32 ? 4 : 2, ws = in.weight_dtype == NS_F32 ? 4 : 2;
  return std::min(std::min(piece_of(in.x, in.x_row, in.D, es), piece_of(y, in.D, in.D, es)),
                  std::min(piece_of(in.weight, 0, in.D, ws), piece_of(in.bias, 0, in.D, ws)));
}

}  // namespace

uint64_t norm_workspace(uint32_t N, uint32_t D) {
  return D ? (uint64_t)back_of(N, D).blocks * 2 * D * sizeof(float) : 0;
}

cudaError_t launch_norm_forward(const ns_norm_inputs &in, void *y, float *mean, float *rstd,
                                cudaStream_t st) {
  NormParams p = params_of(in);
  p.y = y, p.mean = mean, p.rstd = rstd;
  return by_types(in, piece_of_inputs(in, y), [&](auto e, auto w, auto v) {
    return forward_of<decltype(e), decltype(w), decltype(v)::value>(p, st);
  });
}

cudaError_t launch_norm_backward(const ns_norm_inputs &in, const float *mean, const float *rstd,
                                 const void *dy, int64_t dy_row, void *dx, void *dweight,
                                 void *dbias, float *partial, cudaStream_t st) {
  NormParams p = params_of(in);
  p.mean = const_cast<float *>(mean), p.rstd = const_cast<float *>(rstd);
  p.dy = dy, p.dy_row = dy_row, p.y = dx, p.dweight = dweight, p.dbias = dbias;
  p.partial = dweight || dbias ? partial : nullptr;
  const int piece =
      std::min(piece_of_inputs(in, dx), piece_of(dy, dy_row, in.D, in.dtype == NS_F32 ? 4 : 2));
  return by_types(in, piece, [&](auto e, auto w, auto v) {
    return backward_of<decltype(e), decltype(w), decltype(v)::value>(p, st);
  });
}

}  // namespace nsk
