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
// (rows.cuh); a dot product takes a whole row, so that its order depends on nothing but D
// and the rows' alignment.
//
// 32768 x 2560 bf16, 64 experts, k = 8: dispatch 236 us (94 % of the copy's bandwidth),
// combine 229 (95 %), its gradient 415 (100 %).

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "order.h"
#include "rows.cuh"
#include "train.h"

namespace nsk {
namespace {

constexpr int kThreads = 256;

struct ExpertParams {
  uint32_t N, k, E, D;
  // lanes of a unit, spans of a row (rows.cuh) and of a unit, units of a row
  uint32_t lanes, spans, each, slices;
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

// Registers of rows that a lane has under way: 32 of 16-bit rows, eight of which fit in
// four each.  (Eight spans of one choice in pieces of two do not quite fit beside their addresses:
// combine of one choice a token reloads 308 bytes there.)
template <class E, int V>
constexpr int kUnderWay = Oct<E, V>::kPieces * Oct<E, V>::kWords == 4 ? 8 : 4;

// Blocks an SM: as many as have the registers for it (32768 x 2560 bf16, k = 8, backward: two
// 487 us, three 414).
template <class E, int V>
constexpr int kBackBlocks = V == kOct && kUnderWay<E, V> == 8 ? 3 : 2;
constexpr int kCombineBlocks = 2;

// ---- dispatch --------------------------------------------------------------------
// U spans of token n's row, from column `first` on, into the places of its choices.
template <bool kAll, class E, int V, int U>
__device__ __forceinline__ void copy_slice(const ExpertParams &p, const Oct<E, V> (&v)[U],
                                           uint32_t first, uint32_t lanes, const int32_t *place,
                                           uint32_t M) {
  E *to = static_cast<E *>(p.to);
  Oct<E, V> zero;
  clear(zero);
#pragma unroll 2
  for (uint32_t j = 0; j < p.k; ++j) {
    const uint32_t at = (uint32_t)place[j];
    E *row = to + (int64_t)at * p.D;
#pragma unroll
    for (int u = 0; u < U; ++u)
      store_oct<kAll>(row, first + u * lanes * kOct, lanes * V, p.D, at < M ? v[u] : zero);
  }
}
template <bool kAll, class E, int V, int U>
__device__ __forceinline__ void load_slice(const ExpertParams &p, Oct<E, V> (&v)[U], uint32_t n,
                                           uint32_t first, uint32_t lanes) {
  const E *x = static_cast<const E *>(p.x) + (int64_t)n * p.x_row;
#pragma unroll
  for (int u = 0; u < U; ++u)
    load_oct<kAll>(v[u], x, first + u * lanes * kOct, lanes * V, p.D);
}

// A slice of a token a unit: short blocks, whose stores drain while others begin (blocks that
// stay, with the next row under way: 32768 x 2560 bf16, k = 8: 279 us in place of 236).  Its row
// is read before the sort has ended: x was there when the sort's first kernel began.
template <class E, int V, int U, bool kWarp>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const ExpertParams p) {
  const uint32_t lanes = kWarp ? 32 : p.lanes;
  const uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  const uint32_t n = (uint32_t)(unit / p.slices), slice = (uint32_t)(unit % p.slices);
  const uint32_t from = slice * U * lanes * kOct, first = from + threadIdx.x % lanes * V;
  by_all<V, kWarp>(from + U * lanes * kOct, p.D, [&](auto all) {
    constexpr bool kAll = decltype(all)::value;
    Oct<E, V> v[U];
    if (n < p.N) load_slice<kAll>(p, v, n, first, lanes);
    pdl_wait();
    if (n < p.N)
      copy_slice<kAll>(p, v, first, lanes, p.place + (uint64_t)n * p.k, (uint32_t)p.offsets[p.E]);
  });
}

// Few choices: a block a token finds its places by counting the keys below and before
// them, and no sort is needed.  The last block has the offsets.
template <class E, int V, int U>
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
  for (uint32_t unit = threadIdx.x / p.lanes; unit < p.slices; unit += kThreads / p.lanes) {
    const uint32_t first = unit * U * p.lanes * kOct + threadIdx.x % p.lanes * V;
    Oct<E, V> v[U];
    load_slice<false>(p, v, n, first, p.lanes);
    copy_slice<false>(p, v, first, p.lanes, reinterpret_cast<const int32_t *>(count), M);
  }
}

// ---- combine ------------------------------------------------------------------------
// R choices' places and weights; M where there is none.
template <int R>
struct Chosen {
  uint32_t at[R];
  float w[R];
};
template <int R>
__device__ __forceinline__ void load_chosen(Chosen<R> &c, const ExpertParams &p, uint32_t n,
                                            uint32_t j0, uint32_t M) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint64_t s = (uint64_t)n * p.k + j0 + r;
    c.at[r] = j0 + r < p.k ? (uint32_t)p.place[s] : M;
    c.w[r] = p.weights && j0 + r < p.k ? p.weights[s] : 1.0f;
  }
}

// Units of a slice of a token each, one after the other; R choices' rows and U spans of them are
// under way (what hides memory's latency is R U), and the next unit's choices.
template <class E, int V, int R, int U, bool kWarp>
__global__ void __launch_bounds__(kThreads, kCombineBlocks) combine_kernel(const ExpertParams p) {
  const uint32_t M = min((uint32_t)p.offsets[p.E], p.N * p.k);
  const E *from = static_cast<const E *>(p.from);
  const uint32_t lanes = kWarp ? 32 : p.lanes, span = lanes * kOct, step = lanes * V;
  const uint64_t every = (uint64_t)gridDim.x * kThreads / lanes;
  const uint64_t units = (uint64_t)p.N * p.slices;
  uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  Chosen<R> now, next;
  if (unit < units) load_chosen(now, p, (uint32_t)(unit / p.slices), 0, M);
  for (; unit < units; unit += every) {
    const uint32_t n = (uint32_t)(unit / p.slices), slice = (uint32_t)(unit % p.slices);
    if (unit + every < units)
      load_chosen(next, p, (uint32_t)((unit + every) / p.slices), 0, M);
    E *out = static_cast<E *>(p.to) + (int64_t)n * p.D;
    const uint32_t end = min(p.spans, (slice + 1) * p.each);
    for (uint32_t s = slice * p.each; s < end; s += U) {
      const uint32_t first = s * span + threadIdx.x % lanes * V;
      by_all<V, kWarp>((s + U) * span, p.D, [&](auto all) {
        constexpr bool kAll = decltype(all)::value;
        Ch<2> acc[U][kOct / 2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < kOct / 2; ++i) acc[u][i] = {0.0f, 0.0f};
        for (uint32_t j0 = 0; j0 < p.k; j0 += R) {
          if (p.k > R) load_chosen(now, p, n, j0, M);
          Oct<E, V> v[R][U];
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (now.at[r] < M) {
              const E *row = from + (int64_t)now.at[r] * p.from_row;
#pragma unroll
              for (int u = 0; u < U; ++u) load_oct<kAll>(v[r][u], row, first + u * span, step, p.D);
            }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (now.at[r] >= M) continue;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              Ch<2> x[kOct / 2];
              widen(v[r][u], x);
#pragma unroll
              for (int i = 0; i < kOct / 2; ++i)
                acc[u][i] = fma(splat<2>(now.w[r]), x[i], acc[u][i]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (kAll || s + u < end)
            store_oct<kAll>(out, first + u * span, step, p.D, narrow<E, V>(acc[u]));
      });
    }
    now = next;
  }
}

// ---- combine's backward pass -----------------------------------------------------------
// L lanes a choice, T choices at once: neighbouring units are a token's, whose row stays in
// the L1 cache.  T U spans of both rows are under way, and the next choices' places.
template <class E, int V, int T, int U, bool kWarp>
__global__ void __launch_bounds__(kThreads, (kBackBlocks<E, V>))
    combine_backward_kernel(const ExpertParams p) {
  const uint32_t lanes = kWarp ? 32 : p.lanes, span = lanes * kOct, step = lanes * V;
  const uint32_t S = p.N * p.k, lane = threadIdx.x % lanes, groups = kThreads / lanes;
  const uint32_t M = min((uint32_t)p.offsets[p.E], S);
  const uint32_t every = gridDim.x * groups * T;
  Chosen<T> now, next;
  const auto look = [&](Chosen<T> &c, uint64_t b) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const uint64_t s = b + t * groups + threadIdx.x / lanes;
      c.at[t] = s < S ? (uint32_t)p.place[s] : S;
      c.w[t] = s < S && p.weights ? p.weights[s] : 1.0f;
    }
  };
  const uint64_t base = (uint64_t)blockIdx.x * groups * T;  // of the block
  look(now, base);
  // all lanes stay: they add up together
  for (uint64_t b = base; b < S; b += every) {
    look(next, b + every);
    const E *d_out[T];
    Ch<2> dot[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const uint64_t s = b + t * groups + threadIdx.x / lanes;
      d_out[t] = static_cast<const E *>(p.x) + (int64_t)((uint32_t)(s < S ? s : 0) / p.k) * p.x_row;
      dot[t] = {0.0f, 0.0f};
    }
    for (uint32_t c0 = 0; c0 < p.D; c0 += U * span) {
      const uint32_t c = c0 + lane * V;
      by_all<V, kWarp>(c0 + U * span, p.D, [&](auto all) {
        constexpr bool kAll = decltype(all)::value;
        Oct<E, V> a[T][U], y[T][U];
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const E *from = static_cast<const E *>(p.from) + (int64_t)now.at[t] * p.from_row;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (!kAll || now.at[t] >= M) clear(a[t][u]);
            if (!kAll || now.at[t] >= M || !p.d_weights) clear(y[t][u]);
            if (now.at[t] < M) {
              load_oct<kAll>(a[t][u], d_out[t], c + u * span, step, p.D);
              if (p.d_weights) load_oct<kAll>(y[t][u], from, c + u * span, step, p.D);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          if (now.at[t] >= S) continue;
          E *to = static_cast<E *>(p.to) + (int64_t)now.at[t] * p.D;
          const Ch<2> w = splat<2>(now.at[t] < M ? now.w[t] : 1.0f);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            Ch<2> d[kOct / 2], x[kOct / 2];
            widen(a[t][u], d);
            widen(y[t][u], x);
#pragma unroll
            for (int i = 0; i < kOct / 2; ++i) {
              dot[t] = fma(d[i], x[i], dot[t]);
              d[i] = d[i] * w;
            }
            store_oct<kAll>(to, c + u * span, step, p.D, narrow<E, V>(d));
          }
        }
      });
    }
    if (p.d_weights) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const uint64_t s = b + t * groups + threadIdx.x / lanes;
        float sum = dot[t].v[0] + dot[t].v[1];
        for (uint32_t o = lanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (s < S && lane == 0) p.d_weights[s] = sum;
      }
    }
    now = next;
  }
}

// ---- launches ------------------------------------------------------------------------
constexpr uint32_t kSMs = 152;

// Units of `each` spans of a row.
void set_shape(ExpertParams &p, uint32_t each) {
  p.lanes = lanes_for(p.D);
  p.spans = (uint32_t)spans_for(p.D, p.lanes);
  p.each = std::max<uint32_t>(1, each);
  p.slices = (p.spans + p.each - 1) / p.each;
}
// The blocks that all SMs have at once, or as many as there are units for.
uint32_t blocks_for(uint64_t units, uint32_t lanes, uint32_t each_sm) {
  const uint64_t each = kThreads / lanes;
  return (uint32_t)std::min<uint64_t>((units + each - 1) / each, (uint64_t)each_sm * kSMs);
}

// Few choices that each block counts by itself.  A block reads all of the ids, k times from
// shared memory: up to so many comparisons a thread, the sort's two launches cost more (rows of 2048
// bf16, counted and sorted: 64 tokens k = 8 5.0 and 7.8 us, 256 7.0 and 7.7, 512 13.1 and 8.1; 32 of
// k = 32 12.5 and 13.8; 512 of k = 2 4.3 and 6.3; 1024 of k = 1 5.5 and 6.3).  Of one or two choices
// the last ones below the border are slower counted: 1024 of k = 2 8.0 and 6.8, 2048 of k = 1
// 10.3 and 6.9.
bool few(uint64_t N, uint64_t k) { return N * k <= 2048 && N * k * k <= (1 << 14); }

template <class E, int V, int U>
cudaError_t dispatch_by(ExpertParams &p, void *workspace, cudaStream_t st) {
  set_shape(p, U);
  if (few(p.N, p.k)) {
    // counters of a token's choices, or of the experts: alone where no token is, whatever k
    const uint32_t counts = p.N ? std::max(p.k, p.E) : p.E;
    const size_t shared = ((size_t)p.N * p.k + counts + 1) * sizeof(uint32_t);
    ++launch_counter();
    dispatch_few_kernel<E, V, U><<<p.N + 1, kThreads, shared, st>>>(p);
    return cudaGetLastError();
  }
  const cudaError_t e = launch_order_choices({p.ids, nullptr, p.N * p.k, p.E, false}, p.place, p.slots,
                                       p.offsets, workspace, st);
  if (e != cudaSuccess || p.D == 0) return e;
  const uint64_t each = kThreads / p.lanes, blocks = ((uint64_t)p.N * p.slices + each - 1) / each;
  ++launch_counter();
  constexpr bool kFew = U == 1;  // less than a warp's lanes have one span
  pdl_launch(kFew && p.lanes < 32 ? dispatch_kernel<E, V, U, !kFew> : dispatch_kernel<E, V, U, true>,
             dim3((uint32_t)blocks), dim3(kThreads), 0, st, p);
  return cudaGetLastError();
}
template <class E, int V>
cudaError_t dispatch_of(ExpertParams &p, void *workspace, cudaStream_t st) {
  const uint64_t spans = spans_for(p.D, lanes_for(p.D));
  if (spans <= 1) return dispatch_by<E, V, 1>(p, workspace, st);
  if (spans == 2 || kUnderWay<E, V> == 4) return dispatch_by<E, V, 2>(p, workspace, st);
  return dispatch_by<E, V, 4>(p, workspace, st);
}

template <class E, int V, int R>
cudaError_t combine_by(ExpertParams &p, cudaStream_t st) {
  constexpr int U = kUnderWay<E, V> > R ? kUnderWay<E, V> / R : 1;
  // whole rows, or as many units of one as a call of few tokens needs to fill the SMs (2048 columns of
  // bf16, k = 8, whole and in parts: 1 token 5.7 and 2.3 us, 64 6.6 and 2.4, 512 7.2 and 4.2, 2048
  // 15.1 and 15.7, 4096 28.5 both)
  set_shape(p, 1);
  const uint64_t wanted = 32ull * kSMs;
  const uint32_t parts = (uint32_t)std::min<uint64_t>((wanted + p.N - 1) / p.N, (p.spans + U - 1) / U);
  set_shape(p, ((p.spans + parts - 1) / parts + U - 1) / U * U);
  const uint32_t blocks = blocks_for((uint64_t)p.N * p.slices, p.lanes, kCombineBlocks);
  ++launch_counter();
  auto *k = p.lanes == 32 ? combine_kernel<E, V, R, U, true> : combine_kernel<E, V, R, U, false>;
  k<<<blocks, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}
template <class E, int V>
cudaError_t combine_of(ExpertParams &p, cudaStream_t st) {
  if (p.k == 1) return combine_by<E, V, 1>(p, st);
  if (p.k == 2) return combine_by<E, V, 2>(p, st);
  if (p.k <= 4 || kUnderWay<E, V> == 4) return combine_by<E, V, 4>(p, st);
  return combine_by<E, V, kUnderWay<E, V>>(p, st);
}

template <class E, int V, int T, int U>
cudaError_t combine_backward_by(ExpertParams &p, cudaStream_t st) {
  const uint64_t units = ((uint64_t)p.N * p.k + T - 1) / T;
  ++launch_counter();
  constexpr bool kFew = U == 1;  // less than a warp's lanes have one span
  auto *k = kFew && p.lanes < 32 ? combine_backward_kernel<E, V, T, U, !kFew>
                                 : combine_backward_kernel<E, V, T, U, true>;
  k<<<blocks_for(units, p.lanes, kBackBlocks<E, V>), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}
template <class E, int V>
cudaError_t combine_backward_of(ExpertParams &p, cudaStream_t st) {
  constexpr int K = kUnderWay<E, V> / 2;
  set_shape(p, 1);
  if (p.spans <= 1) return combine_backward_by<E, V, K, 1>(p, st);
  if (p.spans == 2) return combine_backward_by<E, V, K / 2, 2>(p, st);
  return combine_backward_by<E, V, 1, K>(p, st);
}

// By the rows' type and the pieces that all of them can be moved by.
template <class F>
cudaError_t by_pieces(int32_t dtype, int piece, F &&call) {
  const auto with = [&](auto e) {
    if (piece == 8) return call(e, std::integral_constant<int, 8>{});
    if (piece == 2) return call(e, std::integral_constant<int, 2>{});
    return call(e, std::integral_constant<int, 1>{});
  };
  if (dtype == NS_F32) return with(float{});
  if (dtype == NS_BF16) return with(__nv_bfloat16{});
  return with(__half{});
}

ExpertParams params_of(const ns_expert_sizes &s) {
  ExpertParams p = {};
  p.N = s.N, p.k = s.k, p.E = s.E, p.D = s.D;
  return p;
}
uint64_t size_of(const ns_expert_sizes &s) { return s.dtype == NS_F32 ? 4 : 2; }

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
  const uint64_t es = size_of(s);
  const int piece = std::min(piece_of(x, x_row, s.D, es), piece_of(rows, s.D, s.D, es));
  return by_pieces(s.dtype, piece, [&](auto e, auto v) {
    return dispatch_of<decltype(e), decltype(v)::value>(p, workspace, st);
  });
}

cudaError_t launch_combine(const ns_expert_sizes &s, const int32_t *place, const int32_t *offsets,
                           const float *weights, const void *rows, int64_t rows_row, void *out,
                           cudaStream_t st) {
  ExpertParams p = params_of(s);
  p.place = const_cast<int32_t *>(place), p.offsets = const_cast<int32_t *>(offsets);
  p.weights = weights, p.from = rows, p.from_row = rows_row, p.to = out;
  const uint64_t es = size_of(s);
  const int piece = std::min(piece_of(rows, rows_row, s.D, es), piece_of(out, s.D, s.D, es));
  return by_pieces(s.dtype, piece, [&](auto e, auto v) {
    return combine_of<decltype(e), decltype(v)::value>(p, st);
  });
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
  const uint64_t es = size_of(s);
  int piece = std::min(piece_of(d_out, d_out_row, s.D, es), piece_of(d_rows, s.D, s.D, es));
  if (d_weights) piece = std::min(piece, piece_of(rows, rows_row, s.D, es));
  return by_pieces(s.dtype, piece, [&](auto e, auto v) {
    return combine_backward_of<decltype(e), decltype(v)::value>(p, st);
  });
}

}  // namespace nsk
