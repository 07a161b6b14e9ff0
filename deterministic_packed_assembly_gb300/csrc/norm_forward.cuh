// Layer norm, forward: see norm.cu.
#pragma once

#include "norm.cuh"

namespace nsk {
namespace {

constexpr int kDirectWarps = 8;  // of a block of rows of up to as many warps

// ---- rows straight from memory -----------------------------------------------------------
// A group of `warps` warps a row; a lane has NB spans of it.
template <class E, int NB, int V>
__global__ void __launch_bounds__(32 * kNormWarps) norm_direct_kernel(const NormParams p) {
  __shared__ float sums[2][kNormWarps];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t group = warp / p.warps, part = warp % p.warps;
  const uint64_t n = (uint64_t)blockIdx.x * (blockDim.x / 32 / p.warps) + group;
  const bool real = n < p.N, there = real && !(p.doc && p.doc[n] < 0);
  constexpr uint32_t span = 32 * kOct, step = 32 * V;
  const uint32_t first = part * NB * span + lane * V;
  const E *x = static_cast<const E *>(p.x) + (int64_t)(real ? n : 0) * p.x_row;
  E *y = static_cast<E *>(p.y) + (int64_t)(real ? n : 0) * p.D;
  const float share = 1.0f / (float)p.D;
  Oct<E, V> v[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    clear(v[i]);
    if (there) load_oct(v[i], x, first + i * span, step, p.D);
  }
  Ch<2> two = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    Ch<2> f[kOct / 2];
    widen(v[i], f);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) two = two + f[j];
  }
  float sum = lanes_sum(two.v[0] + two.v[1], 32);
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
  for (int i = 0; i < NB; ++i) {
    const uint32_t c = first + i * span;
    Ch<2> f[kOct / 2];
    forget(v[i]);
    widen(v[i], f);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      Ch<2> d = f[j] + minus;
      if (!inside<V>(c, step, p.D, 2 * j)) d.v[0] = 0.0f;
      if (!inside<V>(c, step, p.D, 2 * j + 1)) d.v[1] = 0.0f;
      two = fma(d, d, two);
    }
  }
  float square = lanes_sum(two.v[0] + two.v[1], 32);
  if (p.warps > 1) {
    if (lane == 0) sums[1][warp] = square;
    group_sync(group, p.warps);
    square = 0.0f;
    for (uint32_t w = 0; w < p.warps; ++w) square += sums[1][group * p.warps + w];
  }
  const float rstd = __frsqrt_rn(fmaf(square, share, p.eps));
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const uint32_t c = first + i * span;
    if (c >= p.D) break;
    Ch<2> f[kOct / 2], w[kOct / 2], b[kOct / 2];
    load_vector<E, V>(p.weight, p.floats, c, step, p.D, 1.0f, w);
    load_vector<E, V>(p.bias, p.floats, c, step, p.D, 0.0f, b);
    forget(v[i]);
    widen(v[i], f);
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) {
      f[j] = fma((f[j] + minus) * splat<2>(rstd), w[j], b[j]);
      if (!there) f[j] = {0.0f, 0.0f};
    }
    if (real) store_oct(y, c, step, p.D, narrow<E, V>(f));
  }
  if (real && part == 0 && lane == 0) {
    if (p.mean) p.mean[n] = there ? mean : 0.0f;
    if (p.rstd) p.rstd[n] = there ? rstd : 0.0f;
  }
}

// ---- narrow rows ---------------------------------------------------------------------------
// Rows of up to two spans: `lanes` lanes of a warp take M rows at once.
template <class E, int NB, int V>
__global__ void __launch_bounds__(32 * kDirectWarps) norm_narrow_kernel(const NormParams p) {
  constexpr int M = kNormAtOnce<E, NB, V>;
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, per = 32 / p.lanes;
  const uint32_t span = p.lanes * kOct, step = p.lanes * V, first = lane % p.lanes * V;
  const uint64_t n0 = ((uint64_t)blockIdx.x * kDirectWarps + warp) * M * per + lane / p.lanes;
  const float share = 1.0f / (float)p.D;
  Oct<E, V> v[M][NB];
  bool there[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const uint64_t n = n0 + m * per;
    there[m] = n < p.N && !(p.doc && p.doc[n] < 0);
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const E *x = static_cast<const E *>(p.x) + (int64_t)(n0 + m * per) * p.x_row;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      clear(v[m][i]);
      if (there[m]) load_oct(v[m][i], x, first + i * span, step, p.D);
    }
  }
  Ch<2> w[NB][kOct / 2], b[NB][kOct / 2];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    load_vector<E, V>(p.weight, p.floats, first + i * span, step, p.D, 1.0f, w[i]);
    load_vector<E, V>(p.bias, p.floats, first + i * span, step, p.D, 0.0f, b[i]);
  }
  float mean[M], rstd[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    Ch<2> two = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      Ch<2> f[kOct / 2];
      widen(v[m][i], f);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) two = two + f[j];
    }
    mean[m] = two.v[0] + two.v[1];
  }
#pragma unroll
  for (int m = 0; m < M; ++m) mean[m] = lanes_sum(mean[m], p.lanes) * share;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    Ch<2> two = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      Ch<2> f[kOct / 2];
      forget(v[m][i]);
      widen(v[m][i], f);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) {
        Ch<2> d = f[j] + splat<2>(-mean[m]);
        if (!inside<V>(first + i * span, step, p.D, 2 * j)) d.v[0] = 0.0f;
        if (!inside<V>(first + i * span, step, p.D, 2 * j + 1)) d.v[1] = 0.0f;
        two = fma(d, d, two);
      }
    }
    rstd[m] = two.v[0] + two.v[1];
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
    rstd[m] = __frsqrt_rn(fmaf(lanes_sum(rstd[m], p.lanes), share, p.eps));
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const uint64_t n = n0 + m * per;
    if (n >= p.N) break;
    E *y = static_cast<E *>(p.y) + (int64_t)n * p.D;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      Ch<2> f[kOct / 2];
      forget(v[m][i]);
      widen(v[m][i], f);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) {
        f[j] = fma((f[j] + splat<2>(-mean[m])) * splat<2>(rstd[m]), w[i][j], b[i][j]);
        if (!there[m]) f[j] = {0.0f, 0.0f};
      }
      store_oct(y, first + i * span, step, p.D, narrow<E, V>(f));
    }
    if (lane % p.lanes == 0) {
      if (p.mean) p.mean[n] = there[m] ? mean[m] : 0.0f;
      if (p.rstd) p.rstd[n] = there[m] ? rstd[m] : 0.0f;
    }
  }
}

// ---- rows through the ring -----------------------------------------------------------------
// All warps but the last take a batch of R rows together, NB spans each: sums, squares and
// outputs read the batch from shared memory anew, and a batch's sums are exchanged at once.
// kWarps warps at most, kBlocks blocks an SM.
template <class E, int NB, int V, int R, int kWarps, int kBlocks>
__global__ void __launch_bounds__(32 * (kWarps + 1), kBlocks) norm_ring_kernel(const NormParams p) {
  extern __shared__ __align__(128) char shared[];
  NormShared &sh = *reinterpret_cast<NormShared *>(shared);
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t slot = ring_slot(norm_columns(NB, p.warps), sizeof(E));
  start_ring<R>(shared, p.stages, p.warps);
  if (warp == p.warps) {
    produce_rows<E, R, false>(p, shared, shared + kNormRows, slot);
    return;
  }
  constexpr uint32_t kSpan = 32 * kOct, kStep = 32 * V;
  const uint32_t first = warp * NB * kSpan + lane * V;
  const float share = 1.0f / (float)p.D;
  Ch<2> w[NB][kOct / 2], b[NB][kOct / 2];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    load_vector<E, V>(p.weight, p.floats, first + i * kSpan, kStep, p.D, 1.0f, w[i]);
    load_vector<E, V>(p.bias, p.floats, first + i * kSpan, kStep, p.D, 0.0f, b[i]);
  }
  const bool all = (warp + 1) * NB * kSpan <= p.D;  // none of the warp's columns beyond the row
  bool lost = false;
  uint32_t stage = 0, turn = 0;
  for (uint64_t n0 = (uint64_t)blockIdx.x * R; n0 < p.N; n0 += (uint64_t)gridDim.x * R) {
    if (!lost && !barrier_wait(&sh.full[stage], turn & 1)) lost = true;
    if (lost) lose_batch<R>(sh, stage, lane);
    const char *row[R];  // this lane's first columns
    bool there[R];
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t off = first * sizeof(E);
      if constexpr (Oct<E, V>::kBytes < 16)
        off += (uint32_t)reinterpret_cast<uintptr_t>(static_cast<const E *>(p.x) +
                                                     (int64_t)(n0 + r) * p.x_row) & 15u;
      row[r] = ring_row(shared + kNormRows, stage, 0, 1, R, r, slot) + off;
      there[r] = sh.head[stage][r].there;
      // without a branch, so that the batch's rows are computed side by side: what an absent
      // row's place holds comes to nothing
      Ch<2> two = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        Oct<E, V> x;
        Ch<2> f[kOct / 2];
        ring_oct(x, row[r] + i * kSpan * sizeof(E));
        if (!all) only(x, first + i * kSpan, p.D);
        widen(x, f);
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) two = two + f[j];
      }
      v[r] = lost ? norm_lost() : two.v[0] + two.v[1];
    }
    batch_sums<R, kWarps>(v, sh.part[0], p.warps, warp, lane);
    float mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = v[r] * share;
      const Ch<2> minus = splat<2>(-mean[r]);
      Ch<2> two = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t c = first + i * kSpan;
        Oct<E, V> x;
        Ch<2> f[kOct / 2];
        ring_oct(x, row[r] + i * kSpan * sizeof(E));
        widen(x, f);
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) f[j] = f[j] + minus;
        if (!all) {
#pragma unroll
          for (int j = 0; j < kOct; ++j)
            if (!inside<V>(c, kStep, p.D, j)) f[j / 2].v[j & 1] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) two = fma(f[j], f[j], two);
      }
      v[r] = two.v[0] + two.v[1];
    }
    batch_sums<R, kWarps>(v, sh.part[1], p.warps, warp, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t n = n0 + r;
      if (n >= p.N) break;
      const float rstd = __frsqrt_rn(fmaf(v[r], share, p.eps));
      const Ch<2> minus = splat<2>(-mean[r]), scale = splat<2>(rstd);
      E *y = static_cast<E *>(p.y) + (int64_t)n * p.D;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t c = first + i * kSpan;
        Oct<E, V> x, zero;
        Ch<2> f[kOct / 2];
        clear(zero);
        ring_oct(x, row[r] + i * kSpan * sizeof(E));
        widen(x, f);
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) f[j] = fma((f[j] + minus) * scale, w[i][j], b[i][j]);
        x = there[r] ? narrow<E, V>(f) : zero;
        if (all)
          store_all(y + c, x);
        else
          store_oct(y, c, kStep, p.D, x);
      }
      if (threadIdx.x == 0) {
        if (p.mean) p.mean[n] = there[r] ? mean[r] : 0.0f;
        if (p.rstd) p.rstd[n] = there[r] ? rstd : 0.0f;
      }
    }
    __syncwarp();
    if (lane == 0 && !lost) barrier_arrive(&sh.empty[stage]);
    if (++stage == p.stages) stage = 0, ++turn;
  }
}

// ---- rows of any width -----------------------------------------------------------------------
// A block a row, read three times.
template <class E, int V>
__global__ void __launch_bounds__(kWideThreads) norm_wide_kernel(const NormParams p) {
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
    load_vector<E, V>(p.weight, p.floats, c, kStep, D, 1.0f, w);
    load_vector<E, V>(p.bias, p.floats, c, kStep, D, 0.0f, b);
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

// ---- launches -----------------------------------------------------------------------
template <class E, int NB, int V, int R, int kWarps, int kBlocks>
cudaError_t launch_ring(NormParams &p, const NormRing &ring, cudaStream_t st) {
  auto *k = norm_ring_kernel<E, NB, V, R, kWarps, kBlocks>;
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(k), true);
  if (e != cudaSuccess) return e;
  p.stages = ring.stages;
  const uint64_t batches = ((uint64_t)p.N + R - 1) / R;
  const uint32_t blocks = (uint32_t)std::min<uint64_t>(batches, ring.blocks * kNormSMs);
  ++launch_counter();
  k<<<blocks, 32 * (p.warps + 1), ring.shared, st>>>(p);
  return cudaGetLastError();
}
// Batches of four, two or one row, of which the widest rows have the last two; kFew to kWarps
// warps a row.
template <class E, int NB, int V, int kFew, int kWarps, int kBlocks>
cudaError_t ring_of(NormParams &p, cudaStream_t st) {
  constexpr uint32_t kMost = NB > 2 ? 2 : 4, kLeast = kMost / 2;
  const NormRing ring = norm_ring<E, NB, false, kBlocks, kMost, kLeast>(p.warps);
  if constexpr (norm_ring_has<E, NB, false, kFew, kWarps, kBlocks, kMost, kLeast>(kMost))
    if (ring.rows == kMost) return launch_ring<E, NB, V, kMost, kWarps, kBlocks>(p, ring, st);
  if constexpr (norm_ring_has<E, NB, false, kFew, kWarps, kBlocks, kMost, kLeast>(kLeast))
    if (ring.rows == kLeast) return launch_ring<E, NB, V, kLeast, kWarps, kBlocks>(p, ring, st);
  static_assert(!norm_ring_has<E, NB, false, kFew, kWarps, kBlocks, kMost, kLeast>(0), "all have one");
  return cudaErrorInvalidValue;
}

template <class E, int V>
cudaError_t forward_of(NormParams &p, cudaStream_t st) {
  if (p.D > kNormKept) {
    ++launch_counter();
    norm_wide_kernel<E, V><<<p.N, kWideThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  const NormShape s = norm_shape(p.D, false);
  p.lanes = s.lanes, p.warps = s.warps;
  if (p.D <= kNormNarrow) {
    ++launch_counter();
    if (s.nb == 1) {
      const uint32_t rows = kDirectWarps * (32 / p.lanes) * kNormAtOnce<E, 1, V>;
      norm_narrow_kernel<E, 1, V><<<(p.N + rows - 1) / rows, 32 * kDirectWarps, 0, st>>>(p);
    } else {
      const uint32_t rows = kDirectWarps * (32 / p.lanes) * kNormAtOnce<E, 2, V>;
      norm_narrow_kernel<E, 2, V><<<(p.N + rows - 1) / rows, 32 * kDirectWarps, 0, st>>>(p);
    }
    return cudaGetLastError();
  }
  // rows that fill the SMs' rings, else straight from memory: a call of few rows waits for
  // nothing but its own loads (2560 columns of bf16, in the L2 cache: 64 rows 2.7 us, 4.1 through the
  // ring, 608 3.4 and 4.3, 1216 5.5 and 4.8, 4864 19 and 11; 600 columns: 1216 rows 2.9 and
  // 3.8, 2432 4.9 and 4.2).  Wide rows change sides earlier than that: 608 of 5003 floats 7.4
  // and 5.5, of 16384 f16 14.9 and 10.3; 300 of 5003 floats 4.2 and 4.3
  if (p.N > 4 * kNormSMs)
    return s.nb == 1                   ? ring_of<E, 1, V, 3, 5, 5>(p, st)
           : s.nb == 2 && s.warps <= 5 ? ring_of<E, 2, V, 3, 5, 4>(p, st)
           : s.nb == 2                 ? ring_of<E, 2, V, 6, 10, 2>(p, st)
           : s.warps <= 7              ? ring_of<E, 5, V, 5, 7, 2>(p, st)
                                       : ring_of<E, 5, V, 8, kNormWarps, 1>(p, st);
  const uint32_t groups = std::max<uint32_t>(1, kDirectWarps / p.warps);
  const uint32_t threads = groups * p.warps * 32;
  const uint32_t blocks = (uint32_t)(((uint64_t)p.N + groups - 1) / groups);
  ++launch_counter();
  auto *k = s.nb == 1   ? norm_direct_kernel<E, 1, V>
            : s.nb == 2 ? norm_direct_kernel<E, 2, V>
                        : norm_direct_kernel<E, 5, V>;
  k<<<blocks, threads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

template <class E>
cudaError_t norm_forward(NormParams &p, int piece, cudaStream_t st) {
  return norm_by_piece<E>(
      piece, [&](auto v) { return forward_of<E, decltype(v)::value>(p, st); });
}

}  // namespace nsk
