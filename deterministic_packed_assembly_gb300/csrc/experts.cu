// Tokens sorted by expert and back.
//
//   choice s = n k + j of token n has the key ids[s] (E where that is outside [0, E));
//   place = the stable sort's permutation, slots its inverse, offsets[e] = choices before
//   expert e's, M = offsets[E]
//   dispatch:  rows[place[s]] = x[n], 0 from place M on
//   combine:   out[n] = sum_j w[n][j] rows[place[n][j]] over the places below M
//   backward:  d_rows[place] = w d_out[n], d_w[n][j] = <d_out[n], rows[place]>, and for
//              dispatch dx[n] = sum_j d_rows[place], which is combine without weights
//
// Memory bounds all of them, and every pass goes by tokens: their own rows are read
// (or written) once and in order, the sorted rows whole and once each, wherever they lie.
// A choice without an expert has a place behind M, so that the rows there are written
// once too, without a pass of their own.
//
// L lanes take a token and a slice of its columns, eight elements each at a time
// (rows.cuh); a dot product takes a whole row, so that its order depends on nothing but D.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "order.h"
#include "rows.cuh"
#include "train.h"

namespace nsk {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // chunks a lane has under way

struct ExpertParams {
  uint32_t N, k, E, D;
  uint32_t lanes, slices, chunks;  // lanes of a unit, units of a row, chunks of a row
  const int32_t *ids;
  int32_t *place, *slots, *offsets;
  const void *x;       // or d_out
  int64_t x_row;
  const void *from;    // the sorted rows read
  int64_t from_row;
  const float *weights;
  void *to;            // rows, out or d_rows
  float *d_weights;
};

// ---- dispatch --------------------------------------------------------------------
// One slice of token n's row into the places of its choices.
template <class E, bool kWhole>
__device__ __forceinline__ void copy_slice(const ExpertParams &p, uint32_t n, uint32_t slice,
                                           uint32_t lane, const int32_t *place, uint32_t M) {
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  E *to = static_cast<E *>(p.to);
  const uint32_t first = slice * p.lanes * kUnroll + lane;
  Words<E> v[kUnroll];
  if constexpr (kWhole) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (first + u * p.lanes < p.chunks)
        v[u] = load_words<E, true>(x + (int64_t)(first + u * p.lanes) * kChunk);
  }
  Words<E> zero;
#pragma unroll
  for (int i = 0; i < Words<E>::kN; ++i) zero.w[i] = 0;
  for (uint32_t j = 0; j < p.k; ++j) {
    const uint32_t at = (uint32_t)place[j];
    E *row = to + (int64_t)at * p.D;
    const int lead = lead_of<E, kWhole>(row);
    if constexpr (!kWhole) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = (int64_t)(first + u * p.lanes) * kChunk - lead;
        if (at < M && c < p.D) v[u] = load_columns<E, false>(x, c, p.D);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = (int64_t)(first + u * p.lanes) * kChunk - lead;
      if (c < p.D) store_columns<E, kWhole>(row, c, p.D, at < M ? v[u] : zero);
    }
  }
}

// Blocks of kThreads / lanes units: a slice of a token each.
template <class E, bool kWhole>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const ExpertParams p) {
  pdl_wait();
  const uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / p.lanes;
  const uint32_t n = (uint32_t)(unit / p.slices), slice = (uint32_t)(unit % p.slices);
  if (n >= p.N) return;
  copy_slice<E, kWhole>(p, n, slice, threadIdx.x % p.lanes, p.place + (uint64_t)n * p.k,
                        (uint32_t)p.offsets[p.E]);
}

// Few choices: a block a token finds its places by counting the keys below and before
// them, and no sort is needed.  The last block has the offsets.
template <class E, bool kWhole>
__global__ void __launch_bounds__(kThreads) dispatch_few_kernel(const ExpertParams p) {
  extern __shared__ uint32_t key[];  // [S], then what the block counts
  const uint32_t S = p.N * p.k;
  uint32_t *count = key + S;         // [k + 1], or [E + 1]
  const uint32_t n = blockIdx.x, counts = n < p.N ? p.k + 1 : p.E + 1;
  for (uint32_t i = threadIdx.x; i < counts; i += kThreads) count[i] = 0;
  __syncthreads();
  for (uint32_t i0 = 0; i0 < S; i0 += kThreads) {
    const uint32_t i = i0 + threadIdx.x;
    bool there = false;
    if (i < S) {
      const int32_t id = p.ids[i];
      there = id >= 0 && id < (int64_t)p.E;
      key[i] = there ? (uint32_t)id : p.E;
      if (n == p.N) atomicAdd(&count[key[i]], 1u);
    }
    const uint32_t all = __ballot_sync(0xffffffffu, there);
    if (n < p.N && threadIdx.x % 32 == 0) atomicAdd(&count[p.k], __popc(all));
  }
  __syncthreads();
  if (n == p.N) {  // offsets: one warp adds up the experts' counts
    if (threadIdx.x < 32) {
      uint32_t base = 0;
      for (uint32_t e0 = 0; e0 <= p.E; e0 += 32) {
        const uint32_t e = e0 + threadIdx.x;
        const uint32_t c = e <= p.E ? count[e] : 0;
        uint32_t scan = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
          if (threadIdx.x >= (uint32_t)o) scan += v;
        }
        if (e <= p.E) p.offsets[e] = (int32_t)(base + scan - c);
        base += __shfl_sync(0xffffffffu, scan, 31);
      }
    }
    return;
  }
  for (uint32_t j = 0; j < p.k; ++j) {
    const uint32_t s = n * p.k + j, mine = key[s];
    uint32_t ahead = 0;
    for (uint32_t i = threadIdx.x; i < S; i += kThreads)
      ahead += key[i] < mine || (key[i] == mine && i < s);
    ahead = __reduce_add_sync(0xffffffffu, ahead);
    if (threadIdx.x % 32 == 0) atomicAdd(&count[j], ahead);
  }
  __syncthreads();
  for (uint32_t j = threadIdx.x; j < p.k; j += kThreads) {
    p.place[n * p.k + j] = (int32_t)count[j];
    p.slots[count[j]] = (int32_t)(n * p.k + j);
  }
  const uint32_t M = count[p.k];
  for (uint32_t unit = threadIdx.x / p.lanes; unit < p.slices; unit += kThreads / p.lanes)
    copy_slice<E, kWhole>(p, n, unit, threadIdx.x % p.lanes,
                          reinterpret_cast<const int32_t *>(count), M);
}

// ---- combine ------------------------------------------------------------------------
template <class E, bool kWhole>
__global__ void __launch_bounds__(kThreads) combine_kernel(const ExpertParams p) {
  const uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / p.lanes;
  const uint32_t n = (uint32_t)(unit / p.slices), slice = (uint32_t)(unit % p.slices);
  if (n >= p.N) return;
  const uint32_t lane = threadIdx.x % p.lanes;
  const uint32_t M = min((uint32_t)p.offsets[p.E], p.N * p.k);
  const int32_t *place = p.place + (uint64_t)n * p.k;
  const float *weights = p.weights ? p.weights + (uint64_t)n * p.k : nullptr;
  const E *from = static_cast<const E *>(p.from);
  E *out = static_cast<E *>(p.to) + (int64_t)n * p.D;
  const int lead = lead_of<E, kWhole>(out);
  constexpr int kRows = 4;  // rows under way
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t c = (int64_t)(slice * p.lanes * kUnroll + u * p.lanes + lane) * kChunk - lead;
    if (c >= p.D) return;
    float acc[kChunk] = {};
    for (uint32_t j0 = 0; j0 < p.k; j0 += kRows) {
      Words<E> v[kRows];
      float w[kRows];
      bool there[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        there[r] = j0 + r < p.k;
        const uint32_t at = there[r] ? (uint32_t)place[j0 + r] : M;
        there[r] = at < M;
        if (there[r]) {
          v[r] = load_columns<E, kWhole>(from + (int64_t)at * p.from_row, c, p.D);
          w[r] = weights ? weights[j0 + r] : 1.0f;
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (!there[r]) continue;
        float x[kChunk];
        widen<E>(v[r], x);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) acc[i] = fmaf(w[r], x[i], acc[i]);
      }
    }
    store_columns<E, kWhole>(out, c, p.D, narrow<E>(acc));
  }
}

// ---- combine's backward pass -----------------------------------------------------------
// L lanes a choice: neighbouring units are a token's, whose row stays in the L1 cache.
template <class E, bool kWhole>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const ExpertParams p) {
  const uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / p.lanes;
  const uint32_t S = p.N * p.k;
  const bool real = unit < S;  // all lanes stay: they add up together
  const uint32_t s = real ? (uint32_t)unit : S - 1, n = s / p.k;
  const uint32_t lane = threadIdx.x % p.lanes;
  const uint32_t M = min((uint32_t)p.offsets[p.E], S);
  const uint32_t at = (uint32_t)p.place[s];
  const E *d_out = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
  const E *y = static_cast<const E *>(p.from) + (int64_t)at * p.from_row;
  E *to = static_cast<E *>(p.to) + (int64_t)at * p.D;
  const bool there = real && at < M;
  const float w = there && p.weights ? p.weights[s] : there ? 1.0f : 0.0f;
  float dot = 0.0f;
  if (there && (p.d_weights || kWhole)) {
    const uint32_t pieces = (uint32_t)(((uint64_t)p.D + kChunk - 1) / kChunk);
    for (uint32_t q0 = lane; q0 < pieces; q0 += p.lanes * kUnroll) {
      Words<E> a[kUnroll], b[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = (int64_t)(q0 + u * p.lanes) * kChunk;
        if (c < p.D) {
          a[u] = load_columns<E, kWhole>(d_out, c, p.D);
          if (p.d_weights) b[u] = load_columns<E, kWhole>(y, c, p.D);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t c = (int64_t)(q0 + u * p.lanes) * kChunk;
        if (c >= p.D) break;
        float d[kChunk], x[kChunk];
        widen<E>(a[u], d);
        if (p.d_weights) {
          widen<E>(b[u], x);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) dot = fmaf(d[i], x[i], dot);
        }
        if constexpr (kWhole) {
#pragma unroll
          for (int i = 0; i < kChunk; ++i) d[i] *= w;
          store_columns<E, true>(to, c, p.D, narrow<E>(d));
        }
      }
    }
  }
  if (p.d_weights) {
    for (uint32_t o = p.lanes / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (real && lane == 0) p.d_weights[s] = dot;
  }
  if (!real || at >= S || (kWhole && there)) return;
  const int lead = lead_of<E, kWhole>(to);
  for (uint32_t q = lane; q < p.chunks; q += p.lanes) {
    const int64_t c = (int64_t)q * kChunk - lead;
    if (c >= p.D) break;
    float d[kChunk] = {};
    if (there) {
      widen<E>(load_columns<E, kWhole>(d_out, c, p.D), d);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) d[i] *= w;
    }
    store_columns<E, kWhole>(to, c, p.D, narrow<E>(d));
  }
}

// ---- launches ------------------------------------------------------------------------
// Lanes of a unit: as few as hold a row, at most a warp.
void set_shape(ExpertParams &p, bool whole, bool sliced) {
  p.chunks = chunks_of(p.D, whole);
  p.lanes = 1;
  while (p.lanes < 32 && p.lanes < p.chunks) p.lanes *= 2;
  p.slices = sliced ? (p.chunks + p.lanes * kUnroll - 1) / (p.lanes * kUnroll) : 1;
}
uint32_t blocks_of(uint64_t units, uint32_t lanes) {
  const uint32_t each = kThreads / lanes;
  return (uint32_t)((units + each - 1) / each);
}

// Few choices that each block counts by itself.  A block reads all of the ids, k times from
// shared memory: up to so many comparisons a thread, the sort's two launches cost more.
bool few(uint64_t N, uint64_t k) { return N * k <= 2048 && N * k * k <= (1 << 14); }

template <class E>
cudaError_t dispatch_of(ExpertParams &p, void *workspace, cudaStream_t st) {
  const bool whole =
      whole_rows(p.x, p.x_row, p.D, sizeof(E)) && whole_rows(p.to, p.D, p.D, sizeof(E));
  set_shape(p, whole, true);
  if (few(p.N, p.k)) {
    auto *k = whole ? dispatch_few_kernel<E, true> : dispatch_few_kernel<E, false>;
    const size_t shared = (p.N * p.k + std::max(p.k, p.E) + 1) * sizeof(uint32_t);
    ++launch_counter();
    k<<<p.N + 1, kThreads, shared, st>>>(p);
    return cudaGetLastError();
  }
  const cudaError_t e = launch_order_choices({p.ids, nullptr, p.N * p.k, p.E, false}, p.place,
                                             p.slots, p.offsets, workspace, st);
  if (e != cudaSuccess || p.D == 0) return e;
  ++launch_counter();
  pdl_launch(whole ? dispatch_kernel<E, true> : dispatch_kernel<E, false>,
             dim3(blocks_of((uint64_t)p.N * p.slices, p.lanes)), dim3(kThreads), 0, st, p);
  return cudaGetLastError();
}

template <class E>
cudaError_t combine_of(ExpertParams &p, cudaStream_t st) {
  const bool whole =
      whole_rows(p.from, p.from_row, p.D, sizeof(E)) && whole_rows(p.to, p.D, p.D, sizeof(E));
  set_shape(p, whole, true);
  auto *k = whole ? combine_kernel<E, true> : combine_kernel<E, false>;
  ++launch_counter();
  k<<<blocks_of((uint64_t)p.N * p.slices, p.lanes), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <class E>
cudaError_t combine_backward_of(ExpertParams &p, cudaStream_t st) {
  const bool whole = whole_rows(p.x, p.x_row, p.D, sizeof(E)) &&
                     whole_rows(p.from, p.from_row, p.D, sizeof(E)) &&
                     whole_rows(p.to, p.D, p.D, sizeof(E));
  set_shape(p, whole, false);
  auto *k = whole ? combine_backward_kernel<E, true> : combine_backward_kernel<E, false>;
  ++launch_counter();
  k<<<blocks_of((uint64_t)p.N * p.k, p.lanes), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

ExpertParams params_of(const ns_expert_sizes &s) {
  ExpertParams p = {};
  p.N = s.N, p.k = s.k, p.E = s.E, p.D = s.D;
  return p;
}

}  // namespace

uint64_t dispatch_workspace(uint32_t N, uint32_t k, uint32_t E) {
  return few(N, k) ? 0 : order_choices_workspace(N * k, E);
}

cudaError_t launch_dispatch(const ns_expert_sizes &s, const int32_t *ids, const void *x,
                            int64_t x_row, int32_t *place, int32_t *slots, int32_t *offsets,
                            void *rows, void *workspace, cudaStream_t st) {
  ExpertParams p = params_of(s);
  p.ids = ids, p.x = x, p.x_row = x_row;
  p.place = place, p.slots = slots, p.offsets = offsets, p.to = rows;
  switch (s.dtype) {
    case NS_F32: return dispatch_of<float>(p, workspace, st);
    case NS_BF16: return dispatch_of<__nv_bfloat16>(p, workspace, st);
    default: return dispatch_of<__half>(p, workspace, st);
  }
}

cudaError_t launch_combine(const ns_expert_sizes &s, const int32_t *place, const int32_t *offsets,
                           const float *weights, const void *rows, int64_t rows_row, void *out,
                           cudaStream_t st) {
  ExpertParams p = params_of(s);
  p.place = const_cast<int32_t *>(place), p.offsets = const_cast<int32_t *>(offsets);
  p.weights = weights, p.from = rows, p.from_row = rows_row, p.to = out;
  switch (s.dtype) {
    case NS_F32: return combine_of<float>(p, st);
    case NS_BF16: return combine_of<__nv_bfloat16>(p, st);
    default: return combine_of<__half>(p, st);
  }
}

cudaError_t launch_combine_backward(const ns_expert_sizes &s, const int32_t *place,
                                    const int32_t *offsets, const float *weights,
                                    const void *rows, int64_t rows_row, const void *d_out,
                                    int64_t d_out_row, void *d_rows, float *d_weights,
                                    cudaStream_t st) {
  ExpertParams p = params_of(s);
  p.place = const_cast<int32_t *>(place), p.offsets = const_cast<int32_t *>(offsets);
  p.weights = weights, p.from = rows, p.from_row = rows_row;
  p.x = d_out, p.x_row = d_out_row, p.to = d_rows, p.d_weights = d_weights;
  switch (s.dtype) {
    case NS_F32: return combine_backward_of<float>(p, st);
    case NS_BF16: return combine_backward_of<__nv_bfloat16>(p, st);
    default: return combine_backward_of<__half>(p, st);
  }
}

}  // namespace nsk
