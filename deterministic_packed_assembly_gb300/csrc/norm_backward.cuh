// Layer norm, backward: see norm.cu.
#pragma once

#include "norm.cuh"

namespace nsk {
namespace {

constexpr int kNarrowWarps = 8;   // of a block of narrow rows
constexpr int kColumnWarps = 8;    // of 256 columns' sums

// ---- narrow rows ---------------------------------------------------------------------------
// Rows of up to two spans: `lanes` lanes of a warp walk rows, M at once.
template <class E, int NB, int V>
__global__ void __launch_bounds__(32 * kNarrowWarps, 2)
    norm_backward_narrow_kernel(const NormParams p) {
  constexpr int M = kNormAtOnce<E, NB, V>;
  __shared__ float joined[2][NB * 32 * kOct];  // the warps' sums
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32, per = 32 / p.lanes;
  const uint32_t span = p.lanes * kOct, step = p.lanes * V, first = lane % p.lanes * V;
  const float share = 1.0f / (float)p.D;
  Ch<2> w[NB][kOct / 2], dw[NB][kOct / 2], db[NB][kOct / 2];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) dw[i][j] = db[i][j] = {0.0f, 0.0f};
    load_vector<E, V>(p.weight, p.floats, first + i * span, step, p.D, 1.0f, w[i]);
  }
  // a warp's lanes stay together: rows from its first lane's on
  const uint64_t every = (uint64_t)gridDim.x * kNarrowWarps * M * per;
  for (uint64_t n1 = ((uint64_t)blockIdx.x * kNarrowWarps + warp) * M * per; n1 < p.N; n1 += every) {
    const uint64_t n0 = n1 + lane / p.lanes;
    Oct<E, V> x[M][NB], y[M][NB];
    float mean[M], rstd[M], s1[M], s2[M];
    bool there[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint64_t n = n0 + m * per;
      there[m] = n < p.N && !(p.doc && p.doc[n] < 0);
      mean[m] = there[m] ? p.mean[n] : 0.0f, rstd[m] = there[m] ? p.rstd[n] : 0.0f;
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        clear(x[m][i]), clear(y[m][i]);
        if (!there[m]) continue;
        load_oct(x[m][i], static_cast<const E *>(p.x) + (int64_t)(n0 + m * per) * p.x_row,
                 first + i * span, step, p.D);
        load_oct(y[m][i], static_cast<const E *>(p.dy) + (int64_t)(n0 + m * per) * p.dy_row,
                 first + i * span, step, p.D);
      }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      Ch<2> a = {0.0f, 0.0f}, b = a;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        Ch<2> f[kOct / 2], g[kOct / 2];
        widen(x[m][i], f);
        widen(y[m][i], g);
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) {
          const Ch<2> xh = (f[j] + splat<2>(-mean[m])) * splat<2>(rstd[m]), gw = g[j] * w[i][j];
          a = a + gw;
          b = fma(gw, xh, b);
          dw[i][j] = fma(g[j], xh, dw[i][j]);
          db[i][j] = db[i][j] + g[j];
        }
      }
      s1[m] = a.v[0] + a.v[1], s2[m] = b.v[0] + b.v[1];
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
      s1[m] = lanes_sum(s1[m], p.lanes) * -share, s2[m] = lanes_sum(s2[m], p.lanes) * -share;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const uint64_t n = n0 + m * per;
      if (n >= p.N) break;
      E *dx = static_cast<E *>(p.y) + (int64_t)n * p.D;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        Ch<2> f[kOct / 2], g[kOct / 2];
        forget(x[m][i]), forget(y[m][i]);
        widen(x[m][i], f);
        widen(y[m][i], g);
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) {
          const Ch<2> scale = splat<2>(rstd[m]), xh = (f[j] + splat<2>(-mean[m])) * scale;
          f[j] = scale * fma(xh, splat<2>(s2[m]), fma(g[j], w[i][j], splat<2>(s1[m])));
          if (!there[m]) f[j] = {0.0f, 0.0f};
        }
        store_oct(dx, first + i * span, step, p.D, narrow<E, V>(f));
      }
    }
  }
  if (!p.partial) return;
  // lanes that share columns, then warps, in order
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j)
      for (uint32_t o = p.lanes; o < 32; o <<= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          dw[i][j].v[h] += __shfl_xor_sync(kFull, dw[i][j].v[h], o);
          db[i][j].v[h] += __shfl_xor_sync(kFull, db[i][j].v[h], o);
        }
  for (uint32_t g = 0; g < kNarrowWarps; ++g) {
    if (g == warp && lane < p.lanes) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < kOct; ++j) {
          const uint32_t c = first + i * span + j / V * step + j % V;
          const float u = dw[i][j / 2].v[j & 1], v = db[i][j / 2].v[j & 1];
          joined[0][c] = g ? joined[0][c] + u : u;
          joined[1][c] = g ? joined[1][c] + v : v;
        }
    }
    __syncthreads();
  }
  float *to = p.partial + (uint64_t)blockIdx.x * 2 * p.D;
  for (uint32_t c = threadIdx.x; c < p.D; c += blockDim.x)
    to[c] = joined[0][c], to[p.D + c] = joined[1][c];
}

// ---- rows through the ring -----------------------------------------------------------------
// All warps but the last take a batch of R rows together, NB spans each, and keep the sums of
// their columns' dw and db.  The batch is read from shared memory twice: for the rows' two
// sums, exchanged for all R at once, and for dx.
// kWarps warps at most, kBlocks blocks an SM.
template <class E, int NB, int V, int R, int kWarps, int kBlocks>
__global__ void __launch_bounds__(32 * (kWarps + 1), kBlocks)
    norm_backward_ring_kernel(const NormParams p) {
  extern __shared__ __align__(128) char shared[];
  NormShared &sh = *reinterpret_cast<NormShared *>(shared);
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  // the weights of up to three spans stay in registers, those of more in shared memory, a
  // lane's columns beside one another
  constexpr bool kHeld = NB <= 3;
  Ch<2> *kept = reinterpret_cast<Ch<2> *>(shared + kNormRows);
  char *rows = shared + kNormRows + norm_kept(NB, p.warps, true);
  const uint32_t slot = ring_slot(norm_columns(NB, p.warps), sizeof(E));
  start_ring<R>(shared, p.stages, p.warps);
  if (warp == p.warps) {
    produce_rows<E, R, true>(p, shared, rows, slot);
    return;
  }
  constexpr uint32_t kSpan = 32 * kOct, kStep = 32 * V;
  const uint32_t first = warp * NB * kSpan + lane * V;
  const float share = 1.0f / (float)p.D;
  Ch<2> w[kHeld ? NB : 1][kOct / 2], dw[NB][kOct / 2], db[NB][kOct / 2];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) dw[i][j] = db[i][j] = {0.0f, 0.0f};
    Ch<2>(&v)[kOct / 2] = w[kHeld ? i : 0];
    load_vector<E, V>(p.weight, p.floats, first + i * kSpan, kStep, p.D, 1.0f, v);
    if constexpr (!kHeld) {
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) kept[((warp * NB + i) * (kOct / 2) + j) * 32 + lane] = v[j];
    }
  }
  const auto weights = [&](int i) {  // each lane its own
    if constexpr (!kHeld) {
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) w[0][j] = kept[((warp * NB + i) * (kOct / 2) + j) * 32 + lane];
    }
  };
  const bool all = (warp + 1) * NB * kSpan <= p.D;  // none of the warp's columns beyond the row
  bool lost = false;
  uint32_t stage = 0, turn = 0, buffer = 0;
  for (uint64_t n0 = (uint64_t)blockIdx.x * R; n0 < p.N; n0 += (uint64_t)gridDim.x * R) {
    if (!lost && !barrier_wait(&sh.full[stage], turn & 1)) lost = true;
    if (lost) lose_batch<R>(sh, stage, lane);
    const char *xr[R], *gr[R];  // this lane's first columns
    float v[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t xo = first * sizeof(E), go = xo;
      if constexpr (Oct<E, V>::kBytes < 16) {
        xo += (uint32_t)reinterpret_cast<uintptr_t>(static_cast<const E *>(p.x) +
                                                    (int64_t)(n0 + r) * p.x_row) & 15u;
        go += (uint32_t)reinterpret_cast<uintptr_t>(static_cast<const E *>(p.dy) +
                                                    (int64_t)(n0 + r) * p.dy_row) & 15u;
      }
      xr[r] = ring_row(rows, stage, 0, 2, R, r, slot) + xo;
      gr[r] = ring_row(rows, stage, 1, 2, R, r, slot) + go;
      const NormHead head = sh.head[stage][r];
      Ch<2> s1 = {0.0f, 0.0f}, s2 = {0.0f, 0.0f};
      if (head.there) {
        const Ch<2> minus = splat<2>(-head.mean), scale = splat<2>(head.rstd);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          Oct<E, V> x, y;
          Ch<2> f[kOct / 2], g[kOct / 2];
          ring_oct(x, xr[r] + i * kSpan * sizeof(E));
          ring_oct(y, gr[r] + i * kSpan * sizeof(E));
          if (!all) only(x, first + i * kSpan, p.D), only(y, first + i * kSpan, p.D);
          weights(i);
          widen(x, f);
          widen(y, g);
#pragma unroll
          for (int j = 0; j < kOct / 2; ++j) {
            const Ch<2> xh = (f[j] + minus) * scale, gw = g[j] * w[kHeld ? i : 0][j];
            s1 = s1 + gw;
            s2 = fma(gw, xh, s2);
            dw[i][j] = fma(g[j], xh, dw[i][j]);
            db[i][j] = db[i][j] + g[j];
          }
        }
      }
      v[2 * r] = lost ? norm_lost() : s1.v[0] + s1.v[1], v[2 * r + 1] = s2.v[0] + s2.v[1];
    }
    batch_sums<2 * R, kWarps>(v, sh.part[buffer], p.warps, warp, lane);
    buffer ^= 1;  // two buffers: one barrier a batch
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint64_t n = n0 + r;
      if (n >= p.N) break;
      const NormHead head = sh.head[stage][r];
      const Ch<2> minus = splat<2>(-head.mean), scale = splat<2>(head.rstd);
      const Ch<2> m1 = splat<2>(-v[2 * r] * share), m2 = splat<2>(-v[2 * r + 1] * share);
      E *dx = static_cast<E *>(p.y) + (int64_t)n * p.D;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t c = first + i * kSpan;
        Oct<E, V> x, y;
        clear(x);
        if (head.there) {
          Ch<2> f[kOct / 2], g[kOct / 2];
          ring_oct(x, xr[r] + i * kSpan * sizeof(E));
          ring_oct(y, gr[r] + i * kSpan * sizeof(E));
          weights(i);
          widen(x, f);
          widen(y, g);
#pragma unroll
          for (int j = 0; j < kOct / 2; ++j) {
            const Ch<2> xh = (f[j] + minus) * scale;
            f[j] = scale * fma(xh, m2, fma(g[j], w[kHeld ? i : 0][j], m1));
          }
          x = narrow<E, V>(f);
        }
        if (all)
          store_all(dx + c, x);
        else
          store_oct(dx, c, kStep, p.D, x);
      }
    }
    __syncwarp();
    if (lane == 0 && !lost) barrier_arrive(&sh.empty[stage]);
    if (++stage == p.stages) stage = 0, ++turn;
  }
  if (!p.partial) return;
  float *to = p.partial + (uint64_t)blockIdx.x * 2 * p.D;
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < kOct; ++j) {
      const uint32_t c = first + i * kSpan + j / V * kStep + j % V;
      if (c < p.D)
        to[c] = lost ? norm_lost() : dw[i][j / 2].v[j & 1],
        to[p.D + c] = lost ? norm_lost() : db[i][j / 2].v[j & 1];
    }
}

// ---- rows of any width -----------------------------------------------------------------------
// A block a row of any width, read twice.
template <class E, int V>
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
      load_vector<E, V>(p.weight, p.floats, c, kStep, D, 1.0f, w);
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
    load_vector<E, V>(p.weight, p.floats, c, kStep, D, 1.0f, w);
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

// ---- launches -----------------------------------------------------------------------
template <class E, int NB, int V, int R, int kWarps, int kBlocks>
cudaError_t launch_back_ring(NormParams &p, const NormRing &ring, cudaStream_t st) {
  auto *k = norm_backward_ring_kernel<E, NB, V, R, kWarps, kBlocks>;
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(k), true);
  if (e != cudaSuccess) return e;
  p.stages = ring.stages;
  const uint64_t batches = ((uint64_t)p.N + R - 1) / R;
  p.blocks = (uint32_t)std::min<uint64_t>(batches, ring.blocks * kNormSMs);
  ++launch_counter();
  k<<<p.blocks, 32 * (p.warps + 1), ring.shared, st>>>(p);
  return cudaGetLastError();
}
template <class E, int V>
cudaError_t wide_of(NormParams &p, cudaStream_t st) {
  ++launch_counter();
  norm_backward_wide_kernel<E, V><<<p.N, kWideThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  // blocks of 256 columns: enough to fill the SMs, each with rows for its warps
  const uint32_t spans = (p.D + 32 * kOct - 1) / (32 * kOct);
  const uint64_t most = ((uint64_t)p.N + 4 * kColumnWarps - 1) / (4 * kColumnWarps);
  p.blocks = (uint32_t)std::min<uint64_t>(most, (8 * kNormSMs + spans - 1) / spans);
  ++launch_counter();
  norm_columns_kernel<E, V><<<dim3(spans, p.blocks), 32 * kColumnWarps, 0, st>>>(p);
  return cudaGetLastError();
}

// Batches of kMost rows down to kLeast, or straight from memory where the ring has no room;
// kFew to kWarps warps a row.
template <class E, int NB, int V, int kFew, int kWarps, int kBlocks, uint32_t kMost, uint32_t kLeast>
cudaError_t back_ring_of(NormParams &p, cudaStream_t st) {
  const NormRing ring = norm_ring<E, NB, true, kBlocks, kMost, kLeast>(p.warps);
  if constexpr (norm_ring_has<E, NB, true, kFew, kWarps, kBlocks, kMost, kLeast>(4))
    if (ring.rows == 4) return launch_back_ring<E, NB, V, 4, kWarps, kBlocks>(p, ring, st);
  if constexpr (norm_ring_has<E, NB, true, kFew, kWarps, kBlocks, kMost, kLeast>(2))
    if (ring.rows == 2) return launch_back_ring<E, NB, V, 2, kWarps, kBlocks>(p, ring, st);
  if constexpr (norm_ring_has<E, NB, true, kFew, kWarps, kBlocks, kMost, kLeast>(1))
    if (ring.rows == 1) return launch_back_ring<E, NB, V, 1, kWarps, kBlocks>(p, ring, st);
  return wide_of<E, V>(p, st);
}

template <class E, int NB, int V>
cudaError_t narrow_of(NormParams &p, cudaStream_t st) {
  const uint64_t rows = kNarrowWarps * (32 / p.lanes) * kNormAtOnce<E, NB, V>;
  p.blocks = (uint32_t)std::min<uint64_t>((p.N + rows - 1) / rows, 2 * kNormSMs);
  ++launch_counter();
  norm_backward_narrow_kernel<E, NB, V><<<p.blocks, 32 * kNarrowWarps, 0, st>>>(p);
  return cudaGetLastError();
}

template <class E, int V>
cudaError_t backward_of(NormParams &p, cudaStream_t st) {
  const NormShape s = norm_shape(p.D, true);
  p.lanes = s.lanes, p.warps = s.warps;
  if (p.D <= kNormNarrow)
    return s.nb == 1 ? narrow_of<E, 1, V>(p, st) : narrow_of<E, 2, V>(p, st);
  if (p.D > kNormKept) return wide_of<E, V>(p, st);
  return s.nb == 1 && s.warps <= 5    ? back_ring_of<E, 1, V, 3, 5, 4, 4, 2>(p, st)
         : s.nb == 1 && s.warps <= 10 ? back_ring_of<E, 1, V, 6, 10, 2, 4, 2>(p, st)
         : s.nb == 1                  ? back_ring_of<E, 1, V, 11, kNormWarps, 1, 4, 2>(p, st)
         : s.nb == 2                  ? back_ring_of<E, 2, V, 8, kNormWarps, 1, 4, 1>(p, st)
         : s.nb == 3                  ? back_ring_of<E, 3, V, 11, kNormWarps, 1, 2, 1>(p, st)
                                      : back_ring_of<E, 5, V, 10, kNormWarps, 1, 1, 1>(p, st);
}

}  // namespace

template <class E>
cudaError_t norm_backward(NormParams &p, int piece, cudaStream_t st) {
  return norm_by_piece<E>(
      piece, [&](auto v) { return backward_of<E, decltype(v)::value>(p, st); });
}

}  // namespace nsk
