// Rows of a table at a batch's tokens, and the table's gradient.
//
//   y[n] = scale table[t_n],  dtable[v] = scale sum of dy[n] over the n with t_n = v
//
// where a position with doc < 0 or a token outside [0, V) has y = 0 and no gradient.
//
// Memory bounds both.  The gradient has V rows, of which a batch touches few, while a
// few tokens make up much of a batch: the positions are sorted by token (order.cu, so
// that sums have a fixed order and every row is written once), and the order is cut into
// tiles of 32 positions whatever the tokens.  A warp takes a tile's 256 columns; it writes
// the rows of the tokens that begin in its tile, and reads up to 31 positions on for the
// last one.  A token of more positions than that, across tiles, leaves 32-bit sums of each
// tile, which the last kernel adds up, in the tiles' order.  The rows of tokens that are
// not there are filled with 0 by the same launch.
//
// 8 x 4096 tokens of 128256 x 2560 bf16: lookup 40 us (86 % of the copy's bandwidth),
// gradient 140 (87 %), of which the sort 17 and the join 6.  (Rows of 0 filled beside the
// sort's kernels slowed those by as much: 143.)  Many positions of narrow rows are far from that:
// 131072 of 50257 x 512 bf16 83 us of 27, five launches one after the other (by themselves 4, 22 and
// 7 of the sort, 37 of the sums, of which a warp has one tile with nothing of the next under
// way, 9 of the join); 4096 of 32000 x 300 24 of 6 (3, 6, 5, 15, 5).  Partial sums have 256 columns
// a tile at least, and a tile has a whole warp's lanes, whatever the row.

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
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kTile = 32;                 // positions of a tile
constexpr uint32_t kSlice = 32 * kOct;         // columns of a warp
constexpr uint32_t kBefore = 0xffffffffu, kBehind = 0xfffffffeu;

struct EmbedParams {
  const void *tokens;
  const int32_t *doc;
  uint32_t N, V, D;
  int32_t wide;
  float scale;
  // forward
  const void *table;
  int64_t table_row;
  void *y;
  uint32_t lanes, slices;
  // backward
  const void *dy;
  int64_t dy_row;
  void *dtable;
  const Sorted *sorted;
  const uint8_t *used;
  uint32_t *counter;      // tiles in `open`
  uint32_t *open;         // tiles whose last token goes on beyond the next tile's reach
  float *head, *tail;     // [tiles][slices * kSlice]: a tile's sums of the token before it, of
                          // the one that goes on
  uint32_t tiles, sum_blocks;
};

// ---- forward ------------------------------------------------------------------------
// U spans of a position's row a unit: short blocks, whose stores drain while others begin
// (blocks that stay, with the next token under way: 32768 x 2560 bf16 47 us in place of 40).
template <class W, class E, int V, int U, bool kWarp>
__global__ void __launch_bounds__(kThreads) embed_kernel(const EmbedParams p) {
  const uint32_t lanes = kWarp ? 32 : p.lanes, span = lanes * kOct, step = lanes * V;
  const uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  const uint32_t n = (uint32_t)(unit / p.slices), slice = (uint32_t)(unit % p.slices);
  if (n >= p.N) return;
  const int64_t t = p.wide ? static_cast<const int64_t *>(p.tokens)[n]
                           : static_cast<const int32_t *>(p.tokens)[n];
  const bool there = t >= 0 && t < (int64_t)p.V && !(p.doc && p.doc[n] < 0);
  const uint32_t from = slice * U * span, first = from + threadIdx.x % lanes * V;
  const W *row = static_cast<const W *>(p.table) + (there ? t : 0) * p.table_row;
  E *y = static_cast<E *>(p.y) + (int64_t)n * p.D;
  by_all<V, kWarp>(from + U * span, p.D, [&](auto all) {
    constexpr bool kAll = decltype(all)::value;
    Oct<W, V> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!kAll || !there) clear(v[u]);
      if (there) load_oct<kAll>(v[u], row, first + u * span, step, p.D);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Ch<2> x[kOct / 2];
      widen(v[u], x);
#pragma unroll
      for (int i = 0; i < kOct / 2; ++i) x[i] = x[i] * splat<2>(there ? p.scale : 0.0f);
      store_oct<kAll>(y, first + u * span, step, p.D, narrow<E, V>(x));
    }
  });
}

// Narrow rows: T positions at once (131072 x 512 bf16: 35 us one at a time, 29 two).
template <class W, class E, int V, int T, int U, bool kWarp>
__global__ void __launch_bounds__(kThreads) embed_narrow_kernel(const EmbedParams p) {
  const uint32_t lanes = kWarp ? 32 : p.lanes, span = lanes * kOct, step = lanes * V;
  const uint64_t unit = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  const uint64_t n0 = unit / p.slices * T;
  const uint32_t slice = (uint32_t)(unit % p.slices);
  if (n0 >= p.N) return;
  int64_t id[T];
  bool there[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const uint64_t n = n0 + t;
    id[t] = -1;
    if (n < p.N)
      id[t] = p.wide ? static_cast<const int64_t *>(p.tokens)[n]
                     : static_cast<const int32_t *>(p.tokens)[n];
    there[t] = id[t] >= 0 && id[t] < (int64_t)p.V && !(p.doc && n < p.N && p.doc[n] < 0);
  }
  const uint32_t from = slice * U * span, first = from + threadIdx.x % lanes * V;
  by_all<V, kWarp>(from + U * span, p.D, [&](auto all) {
    constexpr bool kAll = decltype(all)::value;
    Oct<W, V> v[T][U];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const W *row = static_cast<const W *>(p.table) + (there[t] ? id[t] : 0) * p.table_row;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!kAll || !there[t]) clear(v[t][u]);
        if (there[t]) load_oct<kAll>(v[t][u], row, first + u * span, step, p.D);
      }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (n0 + t >= p.N) break;
      E *y = static_cast<E *>(p.y) + (int64_t)(n0 + t) * p.D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Ch<2> x[kOct / 2];
        widen(v[t][u], x);
#pragma unroll
        for (int i = 0; i < kOct / 2; ++i) x[i] = x[i] * splat<2>(there[t] ? p.scale : 0.0f);
        store_oct<kAll>(y, first + u * span, step, p.D, narrow<E, V>(x));
      }
    }
  });
}

// ---- backward --------------------------------------------------------------------------
// 0 to the elements at [a, b), by a block.
template <class W>
__device__ __forceinline__ void fill_zero(uintptr_t a, uintptr_t b) {
  uintptr_t lo = (a + 15) / 16 * 16, hi = b / 16 * 16;
  if (lo > hi) lo = hi = b;
  for (uintptr_t i = a + threadIdx.x * sizeof(W); i < lo; i += kThreads * sizeof(W))
    *reinterpret_cast<W *>(i) = from_f32<W>(0.0f);
  for (uintptr_t i = lo + threadIdx.x * 16; i < hi; i += kThreads * 16)
    *reinterpret_cast<uint4 *>(i) = make_uint4(0, 0, 0, 0);
  for (uintptr_t i = hi + threadIdx.x * sizeof(W); i < b; i += kThreads * sizeof(W))
    *reinterpret_cast<W *>(i) = from_f32<W>(0.0f);
}

// Rows of tokens that are not there, of 32 tokens: runs of them are one stretch of bytes.
template <class W>
__device__ __forceinline__ void zero_rows(const EmbedParams &p, uint32_t part) {
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t v0 = part * 32, rows = min(32u, p.V - v0);
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.dtable);
  const uint64_t bytes = (uint64_t)p.D * sizeof(W);
  uint32_t left = __ballot_sync(0xffffffffu, lane < rows && !p.used[v0 + lane]);
  while (left) {
    const int a = __ffs(left) - 1;
    const uint32_t ones = ~(left >> a);
    const int n = ones ? __ffs(ones) - 1 : 32;  // of the run at a
    fill_zero<W>(at + (v0 + a) * bytes, at + (v0 + a + n) * bytes);
    left &= a + n >= 32 ? 0u : ~0u << (a + n);
  }
}

template <class W, class E, int V>
__global__ void __launch_bounds__(kThreads, 3) embed_sum_kernel(const EmbedParams p) {
  pdl_wait();
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (blockIdx.x >= p.sum_blocks) {
    zero_rows<W>(p, blockIdx.x - p.sum_blocks);
    return;
  }
  const uint64_t unit = (uint64_t)blockIdx.x * kWarps + warp;
  const uint32_t tile = (uint32_t)(unit / p.slices), slice = (uint32_t)(unit % p.slices);
  if (tile >= p.tiles) return;
  // three tiles' keys: the one before, this one, the next
  const uint32_t i0 = tile * kTile, i = i0 + lane;
  uint32_t before = kBefore;
  Sorted cur = {kBehind, 0}, next = {kBehind, 0};
  if (tile) before = p.sorted[i - kTile].key;
  if (i < p.N) cur = p.sorted[i];
  if (i + kTile < p.N) next = p.sorted[i + kTile];
  if (cur.key >= p.V) cur.key = kBehind;
  if (next.key >= p.V) next.key = kBehind;
  constexpr uint32_t kAll = 0xffffffffu;
  const uint32_t k0 = __shfl_sync(kAll, cur.key, 0), k31 = __shfl_sync(kAll, cur.key, 31);
  const uint32_t n0 = __popc(__ballot_sync(kAll, cur.key == k0));
  const uint32_t n31 = __popc(__ballot_sync(kAll, cur.key == k31));
  const uint32_t back = __popc(__ballot_sync(kAll, before == k0));  // positions in the tile before
  const uint32_t on = __popc(__ballot_sync(kAll, next.key == k31));  // and in the next one
  if (k0 == kBehind) return;  // padding comes last
  uint32_t e = 0, end = __popc(__ballot_sync(kAll, cur.key != kBehind));
  uint32_t first_end = 0;     // the positions before it go to `head`
  if (back) {
    if (back + n0 > kTile)
      first_end = n0;
    else
      e = n0;                 // the tile before has them
  }
  bool open = false;          // the last token's sum goes to `tail`
  if (k31 != kBehind && on && !(back && n0 == kTile)) {
    if (n31 + on > kTile)
      open = true;
    else
      end += on;
  }
  // partial sums lie by lanes: a lane's eight columns beside one another
  const uint64_t partial = ((uint64_t)tile * p.slices + slice) * kSlice + lane * kOct;
  const uint32_t col = slice * kSlice + lane * V;
  const E *dy = static_cast<const E *>(p.dy);
  W *dtable = static_cast<W *>(p.dtable);
  Ch<2> acc[kOct / 2];
#pragma unroll
  for (int j = 0; j < kOct / 2; ++j) acc[j] = {0.0f, 0.0f};
  constexpr int kAhead = Oct<E, V>::kPieces * Oct<E, V>::kWords == 4 ? 8 : 4;
  while (e < end) {
    Oct<E, V> v[kAhead];
    uint32_t key[kAhead + 1];
#pragma unroll
    for (int a = 0; a <= kAhead; ++a) {
      const uint32_t x = __shfl_sync(kAll, cur.key, (e + a) & 31);
      const uint32_t y = __shfl_sync(kAll, next.key, (e + a) & 31);
      key[a] = e + a >= end ? kBehind : e + a < kTile ? x : y;
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const uint32_t x = __shfl_sync(kAll, cur.at, (e + a) & 31);
      const uint32_t y = __shfl_sync(kAll, next.at, (e + a) & 31);
      const uint32_t at = e + a < kTile ? x : y;
      if (key[a] != kBehind) load_oct(v[a], dy + (int64_t)at * p.dy_row, col, 32 * V, p.D);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (key[a] == kBehind) continue;
      Ch<2> x[kOct / 2];
      widen(v[a], x);
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) acc[j] = acc[j] + x[j];
      if (key[a + 1] == key[a]) continue;
      // the token's last position here
      const bool to_head = e + a < first_end;
      const bool to_tail = open && e + a + 1 == end && !to_head;
      if (to_head || to_tail) {
        float4 *to = reinterpret_cast<float4 *>((to_head ? p.head : p.tail) + partial);
        to[0] = make_float4(acc[0].v[0], acc[0].v[1], acc[1].v[0], acc[1].v[1]);
        to[1] = make_float4(acc[2].v[0], acc[2].v[1], acc[3].v[0], acc[3].v[1]);
        if (to_tail && slice == 0 && lane == 0) p.open[atomicAdd(p.counter, 1u)] = tile;
      } else {
#pragma unroll
        for (int j = 0; j < kOct / 2; ++j) acc[j] = acc[j] * splat<2>(p.scale);
        store_oct(dtable + (int64_t)key[a] * p.D, col, 32 * V, p.D, narrow<W, V>(acc));
      }
#pragma unroll
      for (int j = 0; j < kOct / 2; ++j) acc[j] = {0.0f, 0.0f};
    }
    e += kAhead;
  }
}

// The tokens across tiles: the tail where one begins and the heads behind it.  A
// block takes one's 256 columns, each warp a run of its tiles; the runs are added in order.
constexpr int kJoinWarps = 16;
template <class W, int V>
__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(const EmbedParams p) {
  pdl_wait();
  __shared__ float sums[kJoinWarps][kSlice];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint64_t units = (uint64_t)*p.counter * p.slices;
  for (uint64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const uint32_t tile = p.open[unit / p.slices], slice = (uint32_t)(unit % p.slices);
    const uint32_t key = p.sorted[tile * kTile + kTile - 1].key;
    uint32_t more = 0;  // tiles that begin with the token
    for (;;) {
      const uint64_t at = (uint64_t)(tile + 1 + more + threadIdx.x) * kTile;
      const int n = __syncthreads_count(at < p.N && p.sorted[at].key == key);
      more += n;
      if (n < 32 * kJoinWarps) break;
    }
    const uint32_t run = (more + kJoinWarps - 1) / kJoinWarps;
    const uint32_t a = min(more, warp * run), b = min(more, a + run);
    const uint64_t step = (uint64_t)p.slices * kSlice, at = (uint64_t)slice * kSlice + lane * kOct;
    float acc[kOct] = {};
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < kOct; ++j) acc[j] = p.tail[tile * step + at + j];
    }
#pragma unroll 8
    for (uint32_t t = a; t < b; ++t) {
      const float4 *from = reinterpret_cast<const float4 *>(p.head + (tile + 1 + t) * step + at);
      const float4 x = from[0], y = from[1];
      acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
      acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
    }
#pragma unroll
    for (int j = 0; j < kOct; ++j) sums[warp][lane + 32 * j] = acc[j];
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int j = 0; j < kOct; ++j) acc[j] += sums[w][lane + 32 * j];
      Ch<2> x[kOct / 2];
#pragma unroll
      for (int j = 0; j < kOct; ++j) x[j / 2].v[j & 1] = acc[j] * p.scale;
      store_oct(static_cast<W *>(p.dtable) + (int64_t)key * p.D, slice * kSlice + lane * V, 32 * V,
                p.D, narrow<W, V>(x));
    }
    __syncthreads();
  }
}

// ---- launches ------------------------------------------------------------------------
uint64_t rounded(uint64_t bytes) { return (bytes + 255) / 256 * 256; }
uint32_t tiles_of(uint32_t N) { return (uint32_t)(((uint64_t)N + kTile - 1) / kTile); }

struct Layout {
  uint64_t sorted, used, counter, open, partial, keys, bytes;
};
Layout layout_of(uint32_t N, uint32_t V, uint32_t D) {
  const uint64_t tiles = tiles_of(N);
  const uint64_t columns = ((uint64_t)D + kSlice - 1) / kSlice * kSlice;
  Layout l = {};
  l.sorted = 0;
  l.used = l.sorted + rounded((uint64_t)N * sizeof(Sorted));
  l.counter = l.used + rounded((uint64_t)V + 16);
  l.open = l.counter + 256;
  l.partial = l.open + rounded(tiles * 4);
  l.keys = l.partial + 2 * tiles * columns * sizeof(float);
  l.bytes = l.keys + rounded(order_tokens_workspace(N, V));
  return l;
}

template <class W, class E, int V, int T, int U>
cudaError_t forward_by(EmbedParams &p, cudaStream_t st) {
  p.slices = (uint32_t)((spans_for(p.D, p.lanes) + U - 1) / U);
  const uint64_t each = kThreads / p.lanes, units = ((uint64_t)p.N + T - 1) / T * p.slices;
  const uint32_t blocks = (uint32_t)((units + each - 1) / each);
  ++launch_counter();
  constexpr bool kFew = U == 1;  // less than a warp's lanes have one span
  if constexpr (T == 1) {
    auto *k = kFew && p.lanes < 32 ? embed_kernel<W, E, V, U, !kFew> : embed_kernel<W, E, V, U, true>;
    k<<<blocks, kThreads, 0, st>>>(p);
  } else {
    auto *k = kFew && p.lanes < 32 ? embed_narrow_kernel<W, E, V, T, U, !kFew>
                                   : embed_narrow_kernel<W, E, V, T, U, true>;
    k<<<blocks, kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}
template <class W, class E, int V>
cudaError_t forward_of(EmbedParams &p, cudaStream_t st) {
  p.lanes = lanes_for(p.D);
  const uint64_t spans = spans_for(p.D, p.lanes);
  if (spans > 2) return forward_by<W, E, V, 1, 4>(p, st);
  // several positions at once only where there are enough to fill the SMs (bf16, 128 columns, one
  // and four at once: 8192 positions 2.3 and 2.6 us, 16384 2.9 both, 131072 12.1 and 8.9; 512
  // columns, one and two: 4096 2.3 and 2.4, 8192 2.95 and 3.15, 131072 30.3 and 29.1)
  if ((uint64_t)p.N * p.lanes < 32ull * 32 * 152)
    return spans == 2 ? forward_by<W, E, V, 1, 2>(p, st) : forward_by<W, E, V, 1, 1>(p, st);
  return spans == 2 ? forward_by<W, E, V, 2, 2>(p, st) : forward_by<W, E, V, 4, 1>(p, st);
}

template <class W, class E, int V>
cudaError_t backward_of(EmbedParams &p, void *workspace, cudaStream_t st) {
  char *ws = static_cast<char *>(workspace);
  const Layout l = layout_of(p.N, p.V, p.D);
  Sorted *sorted = reinterpret_cast<Sorted *>(ws + l.sorted);
  uint8_t *used = reinterpret_cast<uint8_t *>(ws + l.used);
  p.sorted = sorted, p.used = used;
  p.counter = reinterpret_cast<uint32_t *>(ws + l.counter);
  p.open = reinterpret_cast<uint32_t *>(ws + l.open);
  p.slices = (p.D + kSlice - 1) / kSlice;
  p.tiles = tiles_of(p.N);
  p.head = reinterpret_cast<float *>(ws + l.partial);
  p.tail = p.head + (uint64_t)p.tiles * p.slices * kSlice;
  cudaError_t e = launch_order_tokens({p.tokens, p.doc, p.N, p.V, p.wide != 0}, sorted, used,
                                      p.counter, ws + l.keys, st);
  if (e != cudaSuccess) return e;
  p.sum_blocks = (uint32_t)(((uint64_t)p.tiles * p.slices + kWarps - 1) / kWarps);
  const uint32_t zero = (p.V + 31) / 32;
  launch_counter() += 2;
  pdl_launch(embed_sum_kernel<W, E, V>, dim3(p.sum_blocks + zero), dim3(kThreads), 0, st, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const uint64_t most = (uint64_t)p.tiles * p.slices;
  pdl_launch(embed_join_kernel<W, V>, dim3((uint32_t)std::min<uint64_t>(most ? most : 1, 3 * 152)),
             dim3(32 * kJoinWarps), 0, st, p);
  return cudaGetLastError();
}

// By the types of the table and of the rows, and the pieces that both can be moved by.
template <class F>
cudaError_t by_types(const ns_embed_inputs &in, int piece, F &&call) {
  const auto with_rows = [&](auto w, auto e) {
    if (piece == 8) return call(w, e, std::integral_constant<int, 8>{});
    if (piece == 2) return call(w, e, std::integral_constant<int, 2>{});
    return call(w, e, std::integral_constant<int, 1>{});
  };
  const auto with_table = [&](auto w) {
    if (in.dtype == NS_F32) return with_rows(w, float{});
    if (in.dtype == NS_BF16) return with_rows(w, __nv_bfloat16{});
    return with_rows(w, __half{});
  };
  if (in.table_dtype == NS_F32) return with_table(float{});
  if (in.table_dtype == NS_BF16) return with_table(__nv_bfloat16{});
  return with_table(__half{});
}
uint64_t size_of(int32_t dtype) { return dtype == NS_F32 ? 4 : 2; }

EmbedParams params_of(const ns_embed_inputs &in) {
  EmbedParams p = {};
  p.tokens = in.tokens, p.doc = in.doc, p.N = in.N, p.V = in.V, p.D = in.D;
  p.wide = in.ids_64 != 0, p.scale = in.scale;
  return p;
}

}  // namespace

uint64_t embed_workspace(uint32_t N, uint32_t V, uint32_t D) { return layout_of(N, V, D).bytes; }

cudaError_t launch_embed_forward(const ns_embed_inputs &in, const void *table, int64_t table_row,
                                 void *y, cudaStream_t st) {
  EmbedParams p = params_of(in);
  p.table = table, p.table_row = table_row, p.y = y;
  const int piece = std::min(piece_of(table, table_row, in.D, size_of(in.table_dtype)),
                             piece_of(y, in.D, in.D, size_of(in.dtype)));
  return by_types(in, piece, [&](auto w, auto e, auto v) {
    return forward_of<decltype(w), decltype(e), decltype(v)::value>(p, st);
  });
}

cudaError_t launch_embed_backward(const ns_embed_inputs &in, const void *dy, int64_t dy_row,
                                  void *dtable, void *workspace, cudaStream_t st) {
  EmbedParams p = params_of(in);
  p.dy = dy, p.dy_row = dy_row, p.dtable = dtable;
  const int piece = std::min(piece_of(dy, dy_row, in.D, size_of(in.dtype)),
                             piece_of(dtable, in.D, in.D, size_of(in.table_dtype)));
  return by_types(in, piece, [&](auto w, auto e, auto v) {
    return backward_of<decltype(w), decltype(e), decltype(v)::value>(p, workspace, st);
  });
}

}  // namespace nsk
