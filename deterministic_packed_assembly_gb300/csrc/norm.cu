// Layer norm of packed positions, and its gradients.
//
//   m = mean of x, r = 1 / sqrt(mean of (x - m)^2 + eps), xh = (x - m) r, y = xh w + b
//   g = dy w,  dx = r (g - mean of g - xh mean of (g xh))
//   dw = sum of dy xh and db = sum of dy over the positions
//
// Memory bounds both passes: a row is read once and kept in registers, as it lies in
// memory, by as few warps as hold it; the variance is taken from the kept values less
// their mean, so that a mean far from 0 costs no digits.  A lane's columns are the same in
// every row, eight at a time (rows.cuh); where rows begin off a boundary, the results are
// moved along by a shuffle and stored in whole chunks all the same.
//
// Backward a group of warps walks rows and keeps the sums of its columns' dw and db in
// registers; blocks write them out once, and the last kernel adds the blocks' rows in
// order.  Rows of more columns than that (kKept) are read twice by the kernel of dx, the
// second time from the caches, and once more by that of dw and db.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "train.h"

namespace nsk {
namespace {

constexpr uint32_t kSMs = 152;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMostWarps = 16;        // of a row
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

// Eight elements from `by` of 16 on (1 to 7).
template <class E>
__device__ __forceinline__ Words<E> moved(const Words<E> &a, const Words<E> &b, uint32_t by) {
  constexpr int n = Words<E>::kN;
  uint32_t u[2 * n];
#pragma unroll
  for (int i = 0; i < n; ++i) u[i] = a.w[i], u[n + i] = b.w[i];
  const uint32_t off = by * sizeof(E);  // bytes
  if constexpr (n == 8)
    if (off & 16) {
#pragma unroll
      for (int i = 0; i < 2 * n - 4; ++i) u[i] = u[i + 4];
    }
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < n + 2; ++i) u[i] = u[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < n + 1; ++i) u[i] = u[i + 1];
  }
  Words<E> r;
#pragma unroll
  for (int i = 0; i < n; ++i) r.w[i] = (off & 2) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
  return r;
}

// A row of D elements from its lanes' chunks, first + 32 i of each lane; every lane of
// the warp calls it, those without a row with `real` false.
template <class E, int NC, bool kWhole>
__device__ __forceinline__ void store_row(E *row, uint32_t first, uint32_t D, uint32_t lanes,
                                          bool real, const Words<E> (&v)[NC]) {
  const uint32_t lane = threadIdx.x % 32;
  const int lead = lead_of<E, kWhole>(row);
  if (kWhole || __all_sync(kFull, lead == 0)) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int64_t c = (int64_t)(first + 32 * i) * kChunk;
      if (real && c < D) store_columns<E, kWhole>(row, c, D, v[i]);
    }
    return;
  }
  const int cut = (kChunk - lead) % kChunk;  // columns before the row's first boundary
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    Words<E> next;
#pragma unroll
    for (int j = 0; j < Words<E>::kN; ++j) {
      const uint32_t mine = i + 1 < NC && lane == 0 ? v[i + 1 < NC ? i + 1 : i].w[j] : v[i].w[j];
      next.w[j] = __shfl_sync(kFull, mine, (lane + 1) % 32);
    }
    const int64_t c = (int64_t)(first + 32 * i) * kChunk;
    if (!real || c >= D) continue;
    const bool last = lane % lanes == lanes - 1 && i == NC - 1;  // the next chunk is not here
    if (cut == 0) {
      store_columns<E, false>(row, c, D, v[i]);
    } else if (!last && c + cut + kChunk <= D) {
      store_words(row + c + cut, moved<E>(v[i], next, cut));
    } else {
      const int to = (int)min((int64_t)(last ? kChunk : kChunk + cut), D - c);
#pragma unroll
      for (int j = 1; j < 2 * kChunk - 1; ++j)
        if (j >= cut && j < to)
          row[c + j] = j < kChunk ? element(v[i], j) : element(next, j - kChunk);
    }
    if (cut && lane % lanes == 0 && i == 0) {  // before the first boundary of these lanes
#pragma unroll
      for (int j = 0; j < kChunk - 1; ++j)
        if (j < cut && c + j < D) row[c + j] = element(v[0], j);
    }
  }
}

// Eight columns of a weight vector, `otherwise` where there is none.
template <class W, bool kWhole>
__device__ __forceinline__ void load_vector(const void *p, int64_t c, int64_t D, float otherwise,
                                            float (&v)[kChunk]) {
  if (p) {
    widen<W>(load_columns<W, kWhole>(static_cast<const W *>(p), c, D), v);
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) v[j] = otherwise;
  }
}

// ---- forward --------------------------------------------------------------------------
// Rows of `lanes` lanes of a warp, or of `warps` warps; NC chunks a lane.
template <class E, class W, int NC, bool kWhole>
__global__ void __launch_bounds__(32 * kMostWarps) norm_forward_kernel(const NormParams p) {
  __shared__ float sums[2][kMostWarps];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t group = warp / p.warps, part = warp % p.warps;
  const uint32_t groups = blockDim.x / 32 / p.warps, per = 32 / p.lanes;
  const uint64_t n = ((uint64_t)blockIdx.x * groups + group) * per + lane / p.lanes;
  const bool real = n < p.N, there = real && !(p.doc && p.doc[n] < 0);
  const uint32_t first = part * NC * 32 + lane % p.lanes;
  const E *x = static_cast<const E *>(p.x) + (int64_t)(real ? n : 0) * p.x_row;
  E *y = static_cast<E *>(p.y) + (int64_t)(real ? n : 0) * p.D;
  const float share = 1.0f / (float)p.D;
  Words<E> v[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int j = 0; j < Words<E>::kN; ++j) v[i].w[j] = 0;
    const int64_t c = (int64_t)(first + 32 * i) * kChunk;
    if (there && c < p.D) v[i] = load_columns<E, kWhole>(x, c, p.D);
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float f[kChunk];
    widen<E>(v[i], f);
#pragma unroll
    for (int j = 0; j < kChunk; ++j) sum += f[j];
  }
  sum = lanes_sum(sum, p.lanes);
  if (p.warps > 1) {
    if (lane == 0) sums[0][warp] = sum;
    group_sync(group, p.warps);
    sum = 0.0f;
    for (uint32_t w = 0; w < p.warps; ++w) sum += sums[0][group * p.warps + w];
  }
  const float mean = sum * share;
  float square = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t c = (int64_t)(first + 32 * i) * kChunk;
    if (c >= p.D) break;
    float f[kChunk];
    widen<E>(v[i], f);
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const float d = f[j] - mean;
      if (kWhole || c + j < p.D) square = fmaf(d, d, square);
    }
  }
  square = lanes_sum(square, p.lanes);
  if (p.warps > 1) {
    if (lane == 0) sums[1][warp] = square;
    group_sync(group, p.warps);
    square = 0.0f;
    for (uint32_t w = 0; w < p.warps; ++w) square += sums[1][group * p.warps + w];
  }
  const float rstd = __frsqrt_rn(fmaf(square, share, p.eps));
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t c = (int64_t)(first + 32 * i) * kChunk;
    float f[kChunk] = {};
    if (there && c < p.D) {
      float w[kChunk], b[kChunk];
      load_vector<W, kWhole>(p.weight, c, p.D, 1.0f, w);
      load_vector<W, kWhole>(p.bias, c, p.D, 0.0f, b);
      widen<E>(v[i], f);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) f[j] = fmaf((f[j] - mean) * rstd, w[j], b[j]);
    }
    v[i] = narrow<E>(f);
  }
  store_row<E, NC, kWhole>(y, first, p.D, p.lanes, real, v);
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
template <class E, class W>
__global__ void __launch_bounds__(kWideThreads) norm_forward_wide_kernel(const NormParams p) {
  __shared__ float sums[kWideThreads / 32];
  const uint32_t n = blockIdx.x;
  const bool there = !(p.doc && p.doc[n] < 0);
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  E *y = static_cast<E *>(p.y) + (int64_t)n * p.D;
  const int lead = lead_of<E, false>(y);
  const int64_t D = p.D, step = kWideThreads * kChunk;
  const int64_t c0 = (int64_t)threadIdx.x * kChunk - lead;
  const float share = 1.0f / (float)p.D;
  float mean = 0.0f, rstd = 0.0f, sum = 0.0f, f[kChunk];
  if (there) {
    for (int64_t c = c0; c < D; c += step) {
      widen<E>(load_columns<E, false>(x, c, D), f);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) sum += f[j];
    }
    mean = block_sum(sum, sums) * share;
    sum = 0.0f;
    for (int64_t c = c0; c < D; c += step) {
      widen<E>(load_columns<E, false>(x, c, D), f);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const float d = f[j] - mean;
        if (c + j >= 0 && c + j < D) sum = fmaf(d, d, sum);
      }
    }
    rstd = __frsqrt_rn(fmaf(block_sum(sum, sums), share, p.eps));
  }
  for (int64_t c = c0; c < D; c += step) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) f[j] = 0.0f;
    if (there) {
      float w[kChunk], b[kChunk];
      load_vector<W, false>(p.weight, c, D, 1.0f, w);
      load_vector<W, false>(p.bias, c, D, 0.0f, b);
      widen<E>(load_columns<E, false>(x, c, D), f);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) f[j] = fmaf((f[j] - mean) * rstd, w[j], b[j]);
    }
    store_columns<E, false>(y, c, D, narrow<E>(f));
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[n] = mean;
    if (p.rstd) p.rstd[n] = rstd;
  }
}

// ---- backward -----------------------------------------------------------------------
// Groups of `warps` warps (or of `lanes` lanes) walk rows; NC chunks a lane.
constexpr int kBackWarps = 10;  // of a block of rows of up to as many warps

template <class E, class W, int NC, bool kWhole, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const NormParams p) {
  __shared__ float2 sums[2][kThreads / 32];
  extern __shared__ float joined[];  // [2][columns]: the groups' sums
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t group = warp / p.warps, part = warp % p.warps;
  const uint32_t groups = blockDim.x / 32 / p.warps, per = 32 / p.lanes;
  const uint32_t first = part * NC * 32 + lane % p.lanes;
  const float share = 1.0f / (float)p.D;
  float w[NC][kChunk], dw[NC][kChunk], db[NC][kChunk];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int64_t c = (int64_t)(first + 32 * i) * kChunk;
#pragma unroll
    for (int j = 0; j < kChunk; ++j) w[i][j] = dw[i][j] = db[i][j] = 0.0f;
    if (c < p.D) load_vector<W, kWhole>(p.weight, c, p.D, 1.0f, w[i]);
  }
  const uint64_t step = (uint64_t)gridDim.x * groups * per;
  uint32_t turn = 0;
  // a group's lanes stay together: rows from the first lane's on
  for (uint64_t n0 = ((uint64_t)blockIdx.x * groups + group) * per; n0 < p.N; n0 += step) {
    const uint64_t n = n0 + lane / p.lanes;
    const bool real = n < p.N, there = real && !(p.doc && p.doc[n] < 0);
    const E *x = static_cast<const E *>(p.x) + (int64_t)(real ? n : 0) * p.x_row;
    const E *dy = static_cast<const E *>(p.dy) + (int64_t)(real ? n : 0) * p.dy_row;
    Words<E> xv[NC], gv[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
      for (int j = 0; j < Words<E>::kN; ++j) xv[i].w[j] = gv[i].w[j] = 0;
      const int64_t c = (int64_t)(first + 32 * i) * kChunk;
      if (there && c < p.D) {
        xv[i] = load_columns<E, kWhole>(x, c, p.D);
        gv[i] = load_columns<E, kWhole>(dy, c, p.D);
      }
    }
    const float mean = there ? p.mean[n] : 0.0f, rstd = there ? p.rstd[n] : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float f[kChunk], g[kChunk];
      widen<E>(xv[i], f);
      widen<E>(gv[i], g);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const float xh = (f[j] - mean) * rstd, gw = g[j] * w[i][j];
        s1 += gw;
        s2 = fmaf(gw, xh, s2);
        dw[i][j] = fmaf(g[j], xh, dw[i][j]);
        db[i][j] += g[j];
      }
    }
    s1 = lanes_sum(s1, p.lanes), s2 = lanes_sum(s2, p.lanes);
    if (p.warps > 1) {  // two buffers: one barrier a row
      if (lane == 0) sums[turn][warp] = make_float2(s1, s2);
      group_sync(group, p.warps);
      s1 = s2 = 0.0f;
      for (uint32_t k = 0; k < p.warps; ++k) {
        const float2 v = sums[turn][group * p.warps + k];
        s1 += v.x, s2 += v.y;
      }
      turn ^= 1;
    }
    s1 *= share, s2 *= share;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float f[kChunk], g[kChunk];
      widen<E>(xv[i], f);
      widen<E>(gv[i], g);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const float xh = (f[j] - mean) * rstd;
        f[j] = there ? rstd * (fmaf(g[j], w[i][j], -s1) - xh * s2) : 0.0f;
      }
      xv[i] = narrow<E>(f);
    }
    store_row<E, NC, kWhole>(static_cast<E *>(p.y) + (int64_t)(real ? n : 0) * p.D, first, p.D,
                             p.lanes, real, xv);
  }
  if (!p.partial) return;
  // lanes that share columns, then groups that do, in order
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      for (uint32_t o = p.lanes; o < 32; o <<= 1) {
        dw[i][j] += __shfl_xor_sync(kFull, dw[i][j], o);
        db[i][j] += __shfl_xor_sync(kFull, db[i][j], o);
      }
  const uint32_t columns = p.warps * NC * p.lanes * kChunk;
  for (uint32_t g = 0; g < groups; ++g) {
    if (g == group && lane < p.lanes) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          float *a = joined + (first + 32 * i) * kChunk + j, *b = a + columns;
          *a = g ? *a + dw[i][j] : dw[i][j];
          *b = g ? *b + db[i][j] : db[i][j];
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
template <class E, class W>
__global__ void __launch_bounds__(kWideThreads) norm_backward_wide_kernel(const NormParams p) {
  __shared__ float sums[kWideThreads / 32];
  const uint32_t n = blockIdx.x;
  const bool there = !(p.doc && p.doc[n] < 0);
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  const E *dy = static_cast<const E *>(p.dy) + (int64_t)n * p.dy_row;
  E *dx = static_cast<E *>(p.y) + (int64_t)n * p.D;
  const int64_t D = p.D, step = kWideThreads * kChunk;
  const int64_t c0 = (int64_t)threadIdx.x * kChunk - lead_of<E, false>(dx);
  float mean = 0.0f, rstd = 0.0f, s1 = 0.0f, s2 = 0.0f, f[kChunk], g[kChunk], w[kChunk];
  if (there) {
    mean = p.mean[n], rstd = p.rstd[n];
    for (int64_t c = c0; c < D; c += step) {
      widen<E>(load_columns<E, false>(x, c, D), f);
      widen<E>(load_columns<E, false>(dy, c, D), g);
      load_vector<W, false>(p.weight, c, D, 1.0f, w);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const float gw = c + j >= 0 && c + j < D ? g[j] * w[j] : 0.0f;
        s1 += gw;
        s2 = fmaf(gw, (f[j] - mean) * rstd, s2);
      }
    }
    s1 = block_sum(s1, sums) / (float)p.D;
    s2 = block_sum(s2, sums) / (float)p.D;
  }
  for (int64_t c = c0; c < D; c += step) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) f[j] = 0.0f;
    if (there) {
      widen<E>(load_columns<E, false>(x, c, D), f);
      widen<E>(load_columns<E, false>(dy, c, D), g);
      load_vector<W, false>(p.weight, c, D, 1.0f, w);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        const float xh = (f[j] - mean) * rstd;
        f[j] = rstd * (fmaf(g[j], w[j], -s1) - xh * s2);
      }
    }
    store_columns<E, false>(dx, c, D, narrow<E>(f));
  }
}

// Rows y, y + blocks, ... of 256 columns.
template <class E, bool kWhole>
__global__ void __launch_bounds__(32 * kColumnWarps) norm_columns_kernel(const NormParams p) {
  __shared__ float sums[kColumnWarps][2][32 * kChunk];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * kChunk;
  float dw[kChunk] = {}, db[kChunk] = {};
  if (c < p.D) {
#pragma unroll 2
    for (uint64_t n = (uint64_t)blockIdx.y * kColumnWarps + warp; n < p.N;
         n += (uint64_t)gridDim.y * kColumnWarps) {
      if (p.doc && p.doc[n] < 0) continue;
      float f[kChunk], g[kChunk];
      const float mean = p.mean[n], rstd = p.rstd[n];
      widen<E>(load_columns<E, kWhole>(static_cast<const E *>(p.x) + (int64_t)n * p.x_row, c, p.D),
               f);
      widen<E>(
          load_columns<E, kWhole>(static_cast<const E *>(p.dy) + (int64_t)n * p.dy_row, c, p.D), g);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        dw[j] = fmaf(g[j], (f[j] - mean) * rstd, dw[j]);
        db[j] += g[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kChunk; ++j) {
    sums[warp][0][lane * kChunk + j] = dw[j];
    sums[warp][1][lane * kChunk + j] = db[j];
  }
  __syncthreads();
  const uint64_t col = (uint64_t)blockIdx.x * 32 * kChunk + threadIdx.x;
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
uint64_t pieces_of(uint32_t D) { return ((uint64_t)D + kChunk - 1) / kChunk; }
uint32_t lanes_of(uint32_t D) {
  uint32_t lanes = 1;
  while (lanes < 32 && lanes < pieces_of(D)) lanes *= 2;
  return lanes;
}

template <class E, class W, int NC>
cudaError_t launch_forward(const NormParams &p, bool whole, uint32_t threads, uint32_t rows,
                           cudaStream_t st) {
  auto *k = whole ? norm_forward_kernel<E, W, NC, true> : norm_forward_kernel<E, W, NC, false>;
  k<<<(uint32_t)(((uint64_t)p.N + rows - 1) / rows), threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <class E, class W>
cudaError_t forward_of(NormParams &p, cudaStream_t st) {
  const bool whole = whole_rows(p.x, p.x_row, p.D, sizeof(E)) &&
                     whole_rows(p.y, p.D, p.D, sizeof(E)) &&
                     whole_rows(p.weight, 0, p.D, sizeof(W)) &&
                     whole_rows(p.bias, 0, p.D, sizeof(W));
  // a lane keeps up to 40 registers of a row
  constexpr uint32_t kMost = 40 / Words<E>::kN;
  const uint64_t pieces = pieces_of(p.D);
  ++launch_counter();
  if (pieces > 32ull * kMost * kMostWarps) {
    norm_forward_wide_kernel<E, W><<<p.N, kWideThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  p.lanes = lanes_of(p.D);
  p.warps = (uint32_t)((pieces + 32 * kMost - 1) / (32 * kMost));
  const uint32_t nc = (uint32_t)((pieces + 32 * p.warps - 1) / (32 * p.warps));
  const uint32_t groups = std::max<uint32_t>(1, 8 / p.warps);
  const uint32_t threads = groups * p.warps * 32, rows = groups * (32 / p.lanes);
  switch (nc) {
    case 1: return launch_forward<E, W, 1>(p, whole, threads, rows, st);
    case 2: return launch_forward<E, W, 2>(p, whole, threads, rows, st);
    case 3: return launch_forward<E, W, 3>(p, whole, threads, rows, st);
    case 4: return launch_forward<E, W, 4>(p, whole, threads, rows, st);
    case 5: return launch_forward<E, W, 5>(p, whole, threads, rows, st);
    default:
      if constexpr (kMost > 5) {
        if (nc <= 6) return launch_forward<E, W, 6>(p, whole, threads, rows, st);
        if (nc <= 8) return launch_forward<E, W, 8>(p, whole, threads, rows, st);
        return launch_forward<E, W, 10>(p, whole, threads, rows, st);
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
  if (D > kKept) {
    // blocks of 256 columns: enough to fill the SMs, each with rows for its warps
    const uint64_t columns = (pieces_of(D) + 31) / 32;
    const uint64_t most = ((uint64_t)N + 4 * kColumnWarps - 1) / (4 * kColumnWarps);
    b.across = (uint32_t)std::min<uint64_t>(most, (8 * kSMs + columns - 1) / columns);
    b.blocks = b.across;
    return b;
  }
  const uint32_t pieces = (uint32_t)pieces_of(D);
  b.lanes = lanes_of(D);
  b.warps = std::max<uint32_t>(1, (pieces + 63) / 64);
  b.nc = (pieces + 32 * b.warps - 1) / (32 * b.warps) > 1 ? 2 : 1;
  b.groups = std::max<uint32_t>(1, kBackWarps / b.warps);
  const uint64_t rows = (uint64_t)b.groups * (32 / b.lanes);
  b.blocks = (uint32_t)std::min<uint64_t>(((uint64_t)N + rows - 1) / rows,
                                          b.warps > kBackWarps ? kSMs : 2 * kSMs);
  return b;
}

template <class E, class W, int NC>
cudaError_t launch_backward(const NormParams &p, const Back &b, bool whole, cudaStream_t st) {
  const uint32_t threads = b.groups * b.warps * 32;
  const size_t shared = 2 * sizeof(float) * b.warps * NC * b.lanes * kChunk;
  auto *k = b.warps > kBackWarps
                ? whole ? norm_backward_kernel<E, W, NC, true, 32 * kMostWarps>
                        : norm_backward_kernel<E, W, NC, false, 32 * kMostWarps>
            : whole ? norm_backward_kernel<E, W, NC, true, 32 * kBackWarps>
                    : norm_backward_kernel<E, W, NC, false, 32 * kBackWarps>;
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(k));
  if (e != cudaSuccess) return e;
  ++launch_counter();
  k<<<b.blocks, threads, shared, st>>>(p);
  return cudaGetLastError();
}

template <class E, class W>
cudaError_t backward_of(NormParams &p, cudaStream_t st) {
  const bool in = whole_rows(p.x, p.x_row, p.D, sizeof(E)) &&
                  whole_rows(p.dy, p.dy_row, p.D, sizeof(E));
  const bool whole = in && whole_rows(p.y, p.D, p.D, sizeof(E)) &&
                     whole_rows(p.weight, 0, p.D, sizeof(W));
  const Back b = back_of(p.N, p.D);
  p.lanes = b.lanes, p.warps = b.warps, p.blocks = b.blocks;
  cudaError_t e = cudaSuccess;
  if (p.N && p.D > kKept) {
    ++launch_counter();
    norm_backward_wide_kernel<E, W><<<p.N, kWideThreads, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.partial) return e;
    auto *k = in ? norm_columns_kernel<E, true> : norm_columns_kernel<E, false>;
    ++launch_counter();
    k<<<dim3((uint32_t)((pieces_of(p.D) + 31) / 32), b.across), 32 * kColumnWarps, 0, st>>>(p);
    e = cudaGetLastError();
  } else if (p.N) {
    e = b.nc == 1 ? launch_backward<E, W, 1>(p, b, whole, st)
                  : launch_backward<E, W, 2>(p, b, whole, st);
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

// By the types of the rows and of the weights, which are floats or as the rows.
template <class F>
cudaError_t by_types(const ns_norm_inputs &in, F &&call) {
  if (in.dtype == NS_F32) return call(float{}, float{});
  if (in.dtype == NS_BF16)
    return in.weight_dtype == NS_F32 ? call(__nv_bfloat16{}, float{})
                                     : call(__nv_bfloat16{}, __nv_bfloat16{});
  return in.weight_dtype == NS_F32 ? call(__half{}, float{}) : call(__half{}, __half{});
}

}  // namespace

uint64_t norm_workspace(uint32_t N, uint32_t D) {
  return D ? (uint64_t)back_of(N, D).blocks * 2 * D * sizeof(float) : 0;
}

cudaError_t launch_norm_forward(const ns_norm_inputs &in, void *y, float *mean, float *rstd,
                                cudaStream_t st) {
  NormParams p = params_of(in);
  p.y = y, p.mean = mean, p.rstd = rstd;
  return by_types(in, [&](auto e, auto w) { return forward_of<decltype(e), decltype(w)>(p, st); });
}

cudaError_t launch_norm_backward(const ns_norm_inputs &in, const float *mean, const float *rstd,
                                 const void *dy, int64_t dy_row, void *dx, void *dweight,
                                 void *dbias, float *partial, cudaStream_t st) {
  NormParams p = params_of(in);
  p.mean = const_cast<float *>(mean), p.rstd = const_cast<float *>(rstd);
  p.dy = dy, p.dy_row = dy_row, p.y = dx, p.dweight = dweight, p.dbias = dbias;
  p.partial = dweight || dbias ? partial : nullptr;
  return by_types(in, [&](auto e, auto w) { return backward_of<decltype(e), decltype(w)>(p, st); });
}

}  // namespace nsk
