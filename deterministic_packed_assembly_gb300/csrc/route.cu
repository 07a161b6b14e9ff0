// A router over packed positions: softmax over E logits a token, its k largest,
// per-expert counts, the balance loss, and the logits' gradient.
//
//   loss = E / (k M^2) sum_e counts_e mass_e,  mass_e = sum_n p_ne
//   dl_nj = p_nj (g_j - sum_e p_ne g_e) + the chosen weights' part,
//   g_e = d_loss E / (k M^2) counts_e
//
// Forward, a thread takes a token (or LP threads a token of more than 128 experts):
// its logits lie in shared memory, in groups of S whose maxima it keeps in
// registers.  A choice is the largest group's, found again among that group's S
// logits alone; of equal ones the first group and the first place win.  Then the
// logits are replaced by their exponentials, and the threads turn round: each
// takes four experts and adds their probabilities up over the tile's tokens.  Blocks
// write rows of partial sums and counts, and a second kernel adds them in a fixed
// order (no floating-point atomics: the loss has the same bits every time).
//
// Backward, L lanes take a token, R experts each, in registers; the softmax is computed
// again, which costs less than keeping it.
//
// Forward (262144 x 256 bfloat16, k = 8: 87 us, 1.7 TB/s) a tile's copies, choices and sums
// follow one another, of 17 to 20 warps an SM: DRAM 24 % and 64 % of the issue slots in the
// first kernel, 77 us; a choice costs 4 us.  Backward issue and memory (62 us, 4.7 TB/s, 72 %
// and DRAM 53 %).

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "train.h"

namespace nsk {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kForwardThreads = 128;
constexpr uint32_t kSMs = 152;
constexpr int kTogether = 8;  // blocks of a cluster

struct RouteParams {
  const void *logits;
  int64_t logits_row;
  const int32_t *doc;
  uint32_t N, E, k;
  int32_t normalize;
  int32_t wide;  // bytes of a row that can be moved at once: 16, 8, 4, or 0 for two
  int32_t *ids;
  float *weights;
  // forward
  int32_t dtype;
  uint32_t lanes;   // threads of a token
  float *mass;      // [blocks][E]
  int32_t *chosen;  // [blocks][E]
  int32_t *real;    // [blocks]
  int32_t *counts, *tokens;
  float *loss;
  uint32_t blocks;
  bool together;    // the blocks are one cluster
  // backward
  const float *d_weights, *d_loss;
  void *dlogits;
};

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float balance(uint32_t E, uint32_t k, int32_t M) {
  return M == 0 ? 0.0f : (float)E / (float)k / ((float)M * (float)M);
}

// ---- forward ------------------------------------------------------------------
// A thread's pieces of a tile of `per` pieces a row, kForwardThreads apart: the row
// and the place move on without a division.
template <class E>
struct Walk {
  uint32_t row, at, rows, rest, per;
  const E *from;
  int64_t step, wrap;
  __device__ __forceinline__ Walk(const RouteParams &p, uint64_t n0, uint32_t pieces,
                                  uint32_t size) {
    per = pieces, rows = kForwardThreads / per, rest = kForwardThreads % per;
    row = threadIdx.x / per, at = threadIdx.x % per;
    from = static_cast<const E *>(p.logits) + (int64_t)(n0 + row) * p.logits_row + at * size;
    step = (int64_t)rows * p.logits_row + rest * size;
    wrap = p.logits_row - (int64_t)per * size;
  }
  __device__ __forceinline__ void next() {
    row += rows, at += rest, from += step;
    if (at >= per) at -= per, ++row, from += wrap;
  }
};

// A tile's logits into shared memory as they are: token n0 + row's expert e at row
// `row * lanes + e / SG`, place e % SG.  `tokens` of them are inside the call.  A
// row of 16-bit logits takes the second half of its room of floats, if it has that: its
// thread widens it in place, from the front.
template <class E, int kBytes, int SG, int kPitch, int kAt>
__device__ __forceinline__ void copy_pieces(const RouteParams &p, uint64_t n0, uint32_t tokens,
                                            float *tile) {
  constexpr int kN = kBytes / sizeof(E);
  Walk<E> w(p, n0, p.E / kN, kN);
  if (w.rest == 0) {  // whole rows at a time: a thread stays in its column
    const uint32_t e = w.at * kN;
    float *row = tile + (w.row * p.lanes + e / SG) * kPitch;
    unsigned char *to = reinterpret_cast<unsigned char *>(
        reinterpret_cast<E *>(row + kAt) + e % SG);
    const uint32_t step = w.rows * p.lanes * kPitch * 4;
#pragma unroll 4
    for (uint32_t r = w.row; r < tokens; r += w.rows, to += step, w.from += w.step)
      copy_async<kBytes>(to, w.from);
    return;
  }
  for (; w.row < tokens; w.next()) {
    const uint32_t e = w.at * kN;
    E *row = reinterpret_cast<E *>(tile + (w.row * p.lanes + e / SG) * kPitch + kAt);
    copy_async<kBytes>(row + e % SG, w.from);
  }
}
template <class E, int SG, int kPitch>
__device__ __forceinline__ void load_tile(const RouteParams &p, uint64_t n0, uint32_t tokens,
                                          float *tile) {
  constexpr int kAt = sizeof(E) == 2 && kPitch > SG ? SG / 2 : 0;
  if (p.wide == 16) {
    copy_pieces<E, 16, SG, kPitch, kAt>(p, n0, tokens, tile);
  } else if (p.wide == 8) {
    copy_pieces<E, 8, SG, kPitch, kAt>(p, n0, tokens, tile);
  } else if (p.wide == 4) {
    copy_pieces<E, 4, SG, kPitch, kAt>(p, n0, tokens, tile);
  } else if constexpr (sizeof(E) == 2) {  // no asynchronous copy takes two bytes
    constexpr int kFlight = 8;
    Walk<E> load(p, n0, p.E, 1), store = load;
    while (load.row < tokens) {
      E v[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i, load.next())
        if (load.row < tokens) v[i] = *load.from;
#pragma unroll
      for (int i = 0; i < kFlight; ++i, store.next())
        if (store.row < tokens)
          reinterpret_cast<E *>(tile + (store.row * p.lanes + store.at / SG) * kPitch +
                                kAt)[store.at % SG] = v[i];
    }
  }
  copy_commit();
  copy_wait<0>();
}

template <int S>
__device__ __forceinline__ void load_group(const float *at, float (&v)[S]) {
#pragma unroll
  for (int q = 0; q < S; q += 4) {
    const float4 x = *reinterpret_cast<const float4 *>(at + q);
    v[q] = x.x, v[q + 1] = x.y, v[q + 2] = x.z, v[q + 3] = x.w;
  }
}

__device__ __forceinline__ void load_pairs(const float *at, Ch<2> (&x)[4]) {
  const float4 a = reinterpret_cast<const float4 *>(at)[0],
               b = reinterpret_cast<const float4 *>(at)[1];
  x[0] = {a.x, a.y}, x[1] = {a.z, a.w}, x[2] = {b.x, b.y}, x[3] = {b.z, b.w};
}
template <class E, int S>
__device__ __forceinline__ void load_narrow(const float *at, float (&v)[S]) {
#pragma unroll
  for (int q = 0; q < S; q += 8) {
    Ch<2> x[4];
    widen_chunk<E>(*reinterpret_cast<const uint4 *>(at + q / 2), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[q + i] = x[i / 2].v[i % 2];
  }
}

// Add the probabilities of a thread's n times four experts, kForwardThreads times four
// (whole rows of SG) apart, up over every `parts`-th token.
template <int n, int SG, int kPitch, int kMax>
__device__ __forceinline__ void add_columns(const float *column, const float *inv, uint32_t first,
                                            uint32_t tokens, uint32_t parts, uint32_t lanes,
                                            Ch<2> (&sum)[kMax][2]) {
  const float *at = column + first * lanes * kPitch;
#pragma unroll 4
  for (uint32_t r = first; r < tokens; r += parts, at += parts * lanes * kPitch) {
    const Ch<2> by = splat<2>(inv[r]);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(at + i * (4 * kForwardThreads / SG) * kPitch);
      sum[i][0] = fma(Ch<2>{x.x, x.y}, by, sum[i][0]);
      sum[i][1] = fma(Ch<2>{x.z, x.w}, by, sum[i][1]);
    }
  }
}

// The same of logits that are kept: their exponentials are computed again.  of[r]: minus
// a token's maximum, and what its exponentials are scaled by.
template <class E, int SG, int kPitch>
__device__ __forceinline__ void add_kept(const float *column, const float2 *of, uint32_t first,
                                         uint32_t tokens, uint32_t parts, uint32_t lanes,
                                         Ch<2> (&sum)[2]) {
  const float *at = column + first * lanes * kPitch;
#pragma unroll 4
  for (uint32_t r = first; r < tokens; r += parts, at += parts * lanes * kPitch) {
    const uint2 x = *reinterpret_cast<const uint2 *>(at);
    const float2 f = of[r];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Ch<2> y = (widen_pair<E>(i ? x.y : x.x) + splat<2>(f.x)) * splat<2>(kLog2e);
      sum[i] = fma(Ch<2>{exp2_sfu(y.v[0]), exp2_sfu(y.v[1])}, splat<2>(f.y), sum[i]);
    }
  }
}

// G groups of S experts a thread.  Its row of shared memory is S * G floats and
// four more, an odd number of 16 bytes: eight threads' 16-byte accesses then use
// all banks.  With a 16-bit type for T the logits (of that type) are kept as they are, in
// half the room: 20 warps share an SM in place of 12, and exponentials are computed twice
// (262144 x 256: 86 us, 97 us with floats in shared memory).
template <int S, int G, class T>
__global__ void __launch_bounds__(kForwardThreads, S != 16 ? 5 : sizeof(T) == 2 ? 5 : 3)
    route_forward_kernel(const RouteParams p) {
  constexpr bool kKept = sizeof(T) == 2;
  constexpr int SG = S * G, kPitch = (kKept ? SG / 2 : SG) + 4, kMaxColumns = NS_ROUTE_MAX_EXPERTS / (4 * kForwardThreads);
  extern __shared__ __align__(16) float tile[];
  const uint32_t LP = p.lanes, tokens = kForwardThreads / LP, columns = LP * SG;
  float *inv = tile + kForwardThreads * kPitch;                     // [tokens]
  float2 *of = reinterpret_cast<float2 *>(inv);                     // or this [tokens]
  int *chosen =                                                     // [columns]
      reinterpret_cast<int *>(inv + (kKept ? 2 : 1) * kForwardThreads);
  float *top_x = reinterpret_cast<float *>(chosen + columns);       // [tokens][k]: logit, weight
  int *top_id = reinterpret_cast<int *>(top_x + tokens * p.k);      // [tokens][k]
  // in a cluster, the first block's: the others' sums and counts, and tokens
  float2 *gathered = reinterpret_cast<float2 *>(top_id + tokens * p.k);
  __shared__ int real_tokens, real_of[kTogether];
  if (p.together) cluster_arrive_relaxed();
  else release_dependents();  // the second kernel is there when this one ends
  const uint32_t tid = threadIdx.x, lane = tid & 31, token = tid / LP, lp = tid % LP;
  float *mine = tile + tid * kPitch;
  for (uint32_t e = tid; e < columns; e += kForwardThreads) chosen[e] = 0;
  if (tid == 0) real_tokens = 0;
  // four experts' (or more, 512 apart) sums over every `parts`-th token
  const uint32_t side = columns / 4 < kForwardThreads ? columns / 4 : kForwardThreads;
  const uint32_t parts = kForwardThreads / side, my_part = tid / side;
  Ch<2> sum[kMaxColumns][2];
#pragma unroll
  for (int i = 0; i < kMaxColumns; ++i) sum[i][0] = sum[i][1] = splat<2>(0.0f);
  int counted = 0;
  const uint64_t tiles = ((uint64_t)p.N + tokens - 1) / tokens;
  for (uint64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const uint64_t n0 = t * tokens;
    __syncthreads();  // the last tile is done with
    const uint32_t here = p.N - n0 < tokens ? (uint32_t)(p.N - n0) : tokens;
    // on its way beside the copies
    const int document =
        token < here ? (p.doc ? __ldg(p.doc + n0 + token) : 0) : -1;
    if constexpr (kKept) load_tile<T, SG, kPitch>(p, n0, here, tile);
    else if (p.dtype == NS_F32) load_tile<float, SG, kPitch>(p, n0, here, tile);
    else if (p.dtype == NS_BF16) load_tile<__nv_bfloat16, SG, kPitch>(p, n0, here, tile);
    else load_tile<__half, SG, kPitch>(p, n0, here, tile);
    const bool real = document >= 0;
    __syncthreads();
    // beyond are places beyond the last expert, and all of a token that does not count
    const int used = !real || p.E <= lp * SG ? 0 : (int)min(p.E - lp * SG, (uint32_t)SG);

    // The k largest: by groups.  NaN is below everything (a maximum leaves it out).
    float top[G];
    float m = kNegInf;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float v[S];
      if constexpr (kKept)
        load_narrow<T, S>(mine + g * S / 2, v);
      else if (p.dtype == NS_F32)
        load_group<S>(mine + g * S, v);
      else if (p.dtype == NS_BF16)
        load_narrow<__nv_bfloat16, S>(mine + SG / 2 + g * S / 2, v);
      else
        load_narrow<__half, S>(mine + SG / 2 + g * S / 2, v);
      if (used < SG) {
#pragma unroll
        for (int q = 0; q < S; ++q)
          if (g * S + q >= used) v[q] = kNegInf;
      }
      if constexpr (kKept) {
        if (used < SG) {
#pragma unroll
          for (int q = 0; q < S; q += 8) {
            const Ch<2> x[4] = {{v[q], v[q + 1]}, {v[q + 2], v[q + 3]}, {v[q + 4], v[q + 5]},
                                {v[q + 6], v[q + 7]}};
            *reinterpret_cast<uint4 *>(mine + (g * S + q) / 2) = narrow_chunk<T>(x);
          }
        }
      } else if (used < SG || p.dtype != NS_F32) {
#pragma unroll
        for (int q = 0; q < S; q += 4)
          *reinterpret_cast<float4 *>(mine + g * S + q) =
              make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
      }
      top[g] = kNegInf;
#pragma unroll
      for (int q = 0; q < S; ++q) top[g] = fmaxf(top[g], v[q]);
      m = fmaxf(m, top[g]);
    }
    for (uint32_t o = LP / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float last_x = kNegInf;  // which is never chosen
    int last = 0;  // this thread's last choice
    for (uint32_t j = 0; j < p.k; ++j) {
      float own = top[0];
#pragma unroll
      for (int g = 1; g < G; ++g) own = fmaxf(own, top[g]);
      float best = own;
      for (uint32_t o = LP / 2; o > 0; o >>= 1)
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
      // the first of the token's threads that has it
      bool me = true;
      if (LP > 1) {
        const uint32_t have = __ballot_sync(0xffffffffu, own == best) >> (lane - lp);
        me = (uint32_t)__ffs(have) == lp + 1;
      }
      if (!me) continue;
      if (best == kNegInf) {
        top_id[token * p.k + j] = -1;
        top_x[token * p.k + j] = kNegInf;
        continue;
      }
      int g = 0;
#pragma unroll
      for (int i = G - 1; i > 0; --i)
        if (top[i] == best) g = i;
      if (top[0] == best) g = 0;
      float v[S];
      if constexpr (kKept) load_narrow<T, S>(mine + g * S / 2, v);
      else load_group<S>(mine + g * S, v);
      uint32_t equal = 0;
      float less = kNegInf;
#pragma unroll
      for (int q = 0; q < S; ++q) {
        if (v[q] == best) equal |= 1u << q;
        if (v[q] < best) less = fmaxf(less, v[q]);
      }
      // equal ones up to the last choice were chosen before
      if (best == last_x && last / S == g) equal &= 0xfffffffeu << (last % S);
      last = g * S + __ffs(equal) - 1;
      last_x = best;
      const float left = equal & (equal - 1) ? best : less;
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (i == g) top[i] = left;
      const int id = lp * SG + last;
      top_id[token * p.k + j] = id;
      top_x[token * p.k + j] = best;
      atomicAdd(&chosen[id], 1);
    }

    // Exponentials in the logits' place, and their sum.  The difference is taken
    // before the change of base, which overflows near the type's lowest value.
    const float base = m == kNegInf ? 0.0f : m;
    // The sum is that of every eight experts, and of those by pairs of neighbours: the
    // same whatever the number of threads.
    constexpr int kRun = SG < 64 ? SG : 64;  // not all unrolled: registers
    float s = 0.0f;
#pragma unroll 1
    for (int i0 = 0; i0 < SG; i0 += kRun) {
      float part[kRun / 8];
#pragma unroll
      for (int i = 0; i < kRun; i += 8) {
        Ch<2> x[4], sum;
        float *at = mine + (kKept ? (i0 + i) / 2 : i0 + i);
        if constexpr (kKept) widen_chunk<T>(*reinterpret_cast<const uint4 *>(at), x);
        else load_pairs(at, x);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const Ch<2> y = (x[q] + splat<2>(-base)) * splat<2>(kLog2e);
          x[q] = {exp2_sfu(y.v[0]), exp2_sfu(y.v[1])};
          sum = q == 0 ? x[q] : sum + x[q];
        }
        if constexpr (!kKept) {
          reinterpret_cast<float4 *>(at)[0] =
              make_float4(x[0].v[0], x[0].v[1], x[1].v[0], x[1].v[1]);
          reinterpret_cast<float4 *>(at)[1] =
              make_float4(x[2].v[0], x[2].v[1], x[3].v[0], x[3].v[1]);
        }
        part[i / 8] = sum.v[0] + sum.v[1];
      }
#pragma unroll
      for (int n = 1; n < kRun / 8; n *= 2)
#pragma unroll
        for (int i = 0; i < kRun / 8; i += 2 * n) part[i] += part[i + n];
      s = i0 == 0 ? part[0] : s + part[0];
    }
    static_assert(SG <= 2 * kRun, "the sum of two runs is that of neighbours");
    for (uint32_t o = 1; o < LP; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float by_all = s == 0.0f ? 0.0f : 1.0f / s;
    if (lp == 0) {
      if constexpr (kKept) of[token] = make_float2(-base, by_all);
      else inv[token] = by_all;
      counted += s != 0.0f;
    }
    __syncwarp();  // the token's threads have written their choices
    float total = 0.0f;
    if (p.normalize)  // every thread in the choices' order
      for (uint32_t j = 0; j < p.k; ++j)
        total += exp2_sfu((top_x[token * p.k + j] - base) * kLog2e);
    __syncwarp();  // before the weights take the logits' places
    // a NaN logit is never chosen, but makes s and so the token's weights NaN
    const float by =
        p.normalize ? (total == 0.0f ? 0.0f : 1.0f / total) + (s - s) : by_all;
    for (uint32_t j = lp; j < p.k; j += LP) {
      const float e = exp2_sfu((top_x[token * p.k + j] - base) * kLog2e);
      top_x[token * p.k + j] = top_id[token * p.k + j] < 0 ? 0.0f : e * by;
    }
    __syncthreads();

    for (uint32_t i = tid; i < here * p.k; i += kForwardThreads) {
      p.ids[n0 * p.k + i] = top_id[i];
      p.weights[n0 * p.k + i] = top_x[i];
    }
    const uint32_t e = tid % side * 4;
    const float *column = tile + e / SG * kPitch + (kKept ? e % SG / 2 : e % SG);
    if constexpr (kKept)
#pragma unroll
      for (int i = 0; i < kMaxColumns; ++i) {
        if (4 * kForwardThreads * i < columns)
          add_kept<T, SG, kPitch>(column + i * (4 * kForwardThreads / SG) * kPitch, of, my_part,
                                  tokens, parts, LP, sum[i]);
      }
    else if (columns <= 4 * kForwardThreads)
      add_columns<1, SG, kPitch>(column, inv, my_part, tokens, parts, LP, sum);
    else
      add_columns<2, SG, kPitch>(column, inv, my_part, tokens, parts, LP, sum);
  }
  counted = warp_sum_i32(counted);
  if (lane == 0) atomicAdd(&real_tokens, counted);
  __syncthreads();
  // the parts of an expert's sum, in order
#pragma unroll
  for (int i = 0; i < kMaxColumns; ++i)
    if (4 * (tid % side + i * kForwardThreads) < columns)
      *reinterpret_cast<float4 *>(tile + my_part * columns + 4 * (tid % side + i * kForwardThreads)) =
          make_float4(sum[i][0].v[0], sum[i][0].v[1], sum[i][1].v[0], sum[i][1].v[1]);
  __syncthreads();
  const uint32_t rank = p.together ? cluster_rank() : 0;
  if (p.together) cluster_wait();  // the first block runs
  for (uint32_t e = tid; e < p.E; e += kForwardThreads) {
    float v = tile[e];
    for (uint32_t q = 1; q < parts; ++q) v += tile[q * columns + e];
    if (p.together) {
      remote_store(remote_smem(&gathered[rank * p.E + e], 0),
                   make_float2(v, __int_as_float(chosen[e])));
    } else {
      p.mass[(uint64_t)blockIdx.x * p.E + e] = v;
      p.chosen[(uint64_t)blockIdx.x * p.E + e] = chosen[e];
    }
  }
  if (!p.together) {
    if (tid == 0) p.real[blockIdx.x] = real_tokens;
    return;
  }
  if (tid == 0) remote_store(remote_smem(&real_of[rank], 0), __int_as_float(real_tokens));
  cluster_arrive();
  cluster_wait();
  if (rank != 0) return;
  // few tokens: the first block of the cluster adds everything up
  float part = 0.0f;
  for (uint32_t e = tid; e < p.E; e += kForwardThreads) {
    float v = 0.0f;
    int n = 0;
    for (uint32_t q = 0; q < gridDim.x; ++q) {
      v += gathered[q * p.E + e].x;
      n += __float_as_int(gathered[q * p.E + e].y);
    }
    p.counts[e] = n;
    part += v * (float)n;
  }
  part = group_sum<32>(part);
  if (lane == 0) inv[tid / 32] = part;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kForwardThreads / 32; ++w) part += inv[w];
    int real = 0;
    for (uint32_t q = 0; q < gridDim.x; ++q) real += real_of[q];
    p.tokens[0] = real;
    p.loss[0] = part * balance(p.E, p.k, real);
  }
}

// The blocks' partial sums, added up by one cluster: block c of it takes a
// share of the experts, `width` lanes side by side and the rest of its threads
// down the rows.
constexpr int kFinalThreads = 1024;
constexpr int kFinalBlocks = 8;
__global__ void __launch_bounds__(kFinalThreads) __cluster_dims__(kFinalBlocks, 1, 1)
    route_total_kernel(const RouteParams p) {
  __shared__ float mass[kFinalThreads];
  __shared__ int chosen[kFinalThreads];
  __shared__ float losses[kFinalBlocks];
  __shared__ float parts[kFinalThreads / 32];
  __shared__ int reals[kFinalThreads / 32];
  const uint32_t rank = cluster_rank();
  cluster_arrive();
  pdl_wait();
  const uint32_t share = (p.E + kFinalBlocks - 1) / kFinalBlocks;
  uint32_t width = 1;
  while (width < share) width *= 2;  // at most 128
  const uint32_t col = threadIdx.x % width, first = threadIdx.x / width,
                 rows = kFinalThreads / width, e = rank * share + col;
  float v = 0.0f;
  int n = 0;
  if (col < share && e < p.E) {
#pragma unroll 8
    for (uint32_t b = first; b < p.blocks; b += rows) {
      v += p.mass[(uint64_t)b * p.E + e];
      n += p.chosen[(uint64_t)b * p.E + e];
    }
  }
  mass[threadIdx.x] = v;
  chosen[threadIdx.x] = n;
  int real = 0;
  if (rank == 0)
    for (uint32_t b = threadIdx.x; b < p.blocks; b += kFinalThreads) real += p.real[b];
  real = warp_sum_i32(real);
  if ((threadIdx.x & 31) == 0) reals[threadIdx.x >> 5] = real;
  for (uint32_t half = kFinalThreads / 2; half >= width; half /= 2) {
    __syncthreads();
    if (threadIdx.x < half) {
      mass[threadIdx.x] += mass[threadIdx.x + half];
      chosen[threadIdx.x] += chosen[threadIdx.x + half];
    }
  }
  __syncthreads();
  float part = 0.0f;
  if (threadIdx.x < width && col < share && e < p.E) {
    p.counts[e] = chosen[col];
    part = mass[col] * (float)chosen[col];
  }
  part = group_sum<32>(part);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = part;
  __syncthreads();
  cluster_wait();  // every block has started
  if (threadIdx.x == 0) {
    for (int w = 1; w < kFinalThreads / 32; ++w) part += parts[w];
    remote_store(remote_smem(&losses[rank], 0), part);
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0 && threadIdx.x == 0) {
    for (int w = 1; w < kFinalThreads / 32; ++w) real += reals[w];
    float loss = losses[0];
    for (int r = 1; r < kFinalBlocks; ++r) loss += losses[r];
    p.tokens[0] = real;
    p.loss[0] = loss * balance(p.E, p.k, real);
  }
}

// ---- backward -------------------------------------------------------------------
// A lane's R experts of a token: every L-th one, or (kPairs) pair of 16-bit ones where
// rows can be moved by 4 bytes, so that lanes side by side move what lies side by side,
// whatever the rows' alignment.  (R consecutive ones, by 16 bytes a lane where aligned:
// 262144 x 256 floats 110 us, 97 us so; bfloat16 69 us and 62 us; 250 experts, by 2
// bytes, 310 us and 61 us.)
template <int L, bool kPairs>
struct Places {
  uint32_t first;
  __device__ __forceinline__ explicit Places(uint32_t lane) : first(lane * (kPairs ? 2 : 1)) {}
  static __device__ __forceinline__ uint32_t after(int r) {  // expert r: first + after(r)
    return r / 2 * 2 * L + r % 2 * (kPairs ? 1 : L);
  }
};

// They as they lie in memory, in pairs: one register of 16-bit ones, or two.
template <class E, int L, int R, bool kPairs>
struct Piece {
  using Pair = std::conditional_t<sizeof(E) == 2, uint32_t, float2>;
  Pair x[R / 2];
  // -inf where there is no expert.
  __device__ __forceinline__ void load(const E *src, const Places<L, kPairs> &at, uint32_t experts) {
#pragma unroll
    for (int r = 0; r < R; r += 2) {
      const uint32_t e = at.after(r), i = at.first + e;
      if constexpr (sizeof(E) == 4) {
        x[r / 2] = {i < experts ? src[e] : kNegInf, i + L < experts ? src[e + L] : kNegInf};
      } else {
        const uint32_t none = narrow_pair<E>(splat<2>(kNegInf));
        if constexpr (kPairs) {
          x[r / 2] = i < experts ? *reinterpret_cast<const uint32_t *>(src + e) : none;
        } else {
          const uint16_t *bits = reinterpret_cast<const uint16_t *>(src);
          const uint32_t lo = i < experts ? bits[e] : none & 0xffffu;
          x[r / 2] = lo | (i + L < experts ? (uint32_t)bits[e + L] << 16 : none & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void widen(Ch<2> (&y)[R / 2]) const {
#pragma unroll
    for (int r = 0; r < R / 2; ++r) {
      if constexpr (sizeof(E) == 4) y[r] = {x[r].x, x[r].y};
      else y[r] = widen_pair<E>(x[r]);
    }
  }
};
template <class E, int L, int R, bool kPairs>
__device__ __forceinline__ void store_logits(E *dst, const Places<L, kPairs> &at, uint32_t experts,
                                             const Ch<2> (&d)[R / 2]) {
#pragma unroll
  for (int r = 0; r < R; r += 2) {
    const uint32_t e = at.after(r), i = at.first + e;
    const Ch<2> &y = d[r / 2];
    if constexpr (sizeof(E) == 4) {
      if (i < experts) dst[e] = y.v[0];
      if (i + L < experts) dst[e + L] = y.v[1];
    } else {
      const uint32_t v = narrow_pair<E>(y);
      uint16_t *bits = reinterpret_cast<uint16_t *>(dst);
      if constexpr (kPairs) {
        if (i < experts) *reinterpret_cast<uint32_t *>(dst + e) = v;
      } else {
        if (i < experts) bits[e] = (uint16_t)v;
        if (i + L < experts) bits[e + L] = (uint16_t)(v >> 16);
      }
    }
  }
}

template <class E, int L, int R, bool kPairs, bool kNormalize>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 2 && R == 16 ? 3 : 2)
    route_backward_kernel(const RouteParams p) {
  constexpr int G = 32 / L, kExperts = L * R, kP = R / 2;
  // the weights' part of a token's gradient, 0 but where it has one
  __shared__ __align__(16) float add[kWarps][G][kExperts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / L, gl = lane % L;
  const Places<L, kPairs> mine(gl);
  const uint32_t i0 = mine.first;
  float *my_add = add[warp][group];
  Ch<2> g[kP];
  const float coef = p.d_loss ? p.d_loss[0] * balance(p.E, p.k, p.tokens[0]) : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t e = i0 + mine.after(r);
    g[r / 2].v[r % 2] = p.d_loss && e < p.E ? coef * (float)p.counts[e] : 0.0f;
    my_add[e] = 0.0f;
  }
  __syncwarp();
  const uint32_t step = gridDim.x * kWarps * G;
  const uint64_t n_first = ((uint64_t)blockIdx.x * kWarps + warp) * G + group;
  const E *src = static_cast<const E *>(p.logits) + (int64_t)n_first * p.logits_row + i0;
  E *dst = static_cast<E *>(p.dlogits) + (int64_t)n_first * p.E + i0;
  // a token's document id is read two steps ahead: whether its logits are to be read
  // is known when the step before begins
  auto document = [&](uint64_t n) { return n < p.N ? (p.doc ? __ldg(p.doc + n) : 0) : -1; };
  bool next_real = document(n_first) >= 0;
  int ahead = document(n_first + step);
  Piece<E, L, R, kPairs> next;
  if (next_real) next.load(src, mine, p.E);
  // A lane has one of the token's choices at most, or goes through several.
  const bool one = p.k <= (uint32_t)L;
  int next_id = -1;  // -1: there is no such choice
  float next_w = 0.0f, next_dw = 0.0f;
  auto load_choice = [&](uint64_t n) {
    next_id = -1;
    if (next_real && p.d_weights && one && gl < (int)p.k) {
      const uint32_t at = (uint32_t)n * p.k + gl;  // below 2^31
      next_id = p.ids[at], next_w = p.weights[at], next_dw = p.d_weights[at];
    }
  };
  load_choice(n_first);
  for (uint64_t n0 = n_first - group; n0 < p.N;) {
    const uint64_t n = n0 + group;
    const bool in = n < p.N, real = next_real;
    Ch<2> x[kP];
    next.widen(x);
    if (!real) {
#pragma unroll
      for (int r = 0; r < kP; ++r) x[r] = splat<2>(kNegInf);
    }
    // w = p at the chosen ones: dl_j = w_j dw_j - p_j t at them, t = sum w dw;
    // normalised, w is their own softmax: dl_j = w_j (dw_j - t).
    const int id = next_id;
    const float w = next_w, dw = next_dw;
    n0 += step, src += (int64_t)step * p.logits_row;
    next_real = ahead >= 0;
    ahead = document(n0 + group + step);
    if (next_real) next.load(src, mine, p.E);
    load_choice(n0 + group);
    const uint32_t at = real ? (uint32_t)n * p.k : 0;
    float m = kNegInf;
#pragma unroll
    for (int r = 0; r < kP; ++r) m = fmaxf(m, fmaxf(x[r].v[0], x[r].v[1]));
    m = group_max<L>(m);
    const Ch<2> base = splat<2>(m == kNegInf ? 0.0f : -m);
    Ch<2> s2 = splat<2>(0.0f), dot2 = s2;
#pragma unroll
    for (int r = 0; r < kP; ++r) {
      const Ch<2> y = (x[r] + base) * splat<2>(kLog2e);
      x[r] = {exp2_sfu(y.v[0]), exp2_sfu(y.v[1])};
      s2 = s2 + x[r];
      dot2 = fma(x[r], g[r], dot2);
    }
    // Normalised weights' gradient is the same for dw plus a constant: taken from the
    // first choice's, of the largest weight, dw_j - t loses nothing where they are alike.
    float from = 0.0f;
    if constexpr (kNormalize) from = __shfl_sync(0xffffffffu, dw, group * L);
    float t = id >= 0 ? w * (dw - from) : 0.0f;
    if (p.d_weights && real && !one) {
      if (kNormalize) from = p.d_weights[at];
      for (uint32_t j = gl; j < p.k; j += L)
        if (p.ids[at + j] >= 0) t += p.weights[at + j] * (p.d_weights[at + j] - from);
    }
    float s = s2.v[0] + s2.v[1], dot = dot2.v[0] + dot2.v[1];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
      t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    const float inv = s == 0.0f ? 0.0f : rcp_sfu(s), mean = kNormalize ? t : 0.0f;
    if (p.d_weights) {
      if (one) {
        if (id >= 0 && id < (int)p.E) my_add[id] = w * ((dw - from) - mean);
      } else if (real) {
        for (uint32_t j = gl; j < p.k; j += L) {
          const int e = p.ids[at + j];
          if (e >= 0 && e < (int)p.E)
            my_add[e] = p.weights[at + j] * ((p.d_weights[at + j] - from) - mean);
        }
      }
      __syncwarp();
    }
    dot = fmaf(dot, inv, kNormalize ? 0.0f : t);
    const Ch<2> inv2 = splat<2>(inv), minus = splat<2>(-dot);
#pragma unroll
    for (int r = 0; r < kP; ++r) {
      const float *a = my_add + i0 + mine.after(2 * r);
      const Ch<2> v = kPairs ? *reinterpret_cast<const Ch<2> *>(a) : Ch<2>{a[0], a[L]};
      x[r] = fma(x[r] * inv2, g[r] + minus, v);
    }
    if (s == 0.0f) {  // the token counts for nothing
#pragma unroll
      for (int r = 0; r < kP; ++r) x[r] = splat<2>(0.0f);
    }
    if (in) store_logits<E, L, R, kPairs>(dst, mine, p.E, x);
    dst += (int64_t)step * p.E;
    if (p.d_weights) {
      __syncwarp();
      if (one) {
        if (id >= 0 && id < (int)p.E) my_add[id] = 0.0f;
      } else if (real) {
        for (uint32_t j = gl; j < p.k; j += L) {
          const int e = p.ids[at + j];
          if (e >= 0 && e < (int)p.E) my_add[e] = 0.0f;
        }
      }
      __syncwarp();
    }
  }
}

// The forward kernel's groups and threads a token.  With tokens enough to fill the GPU: up
// to 64 experts a thread, in groups of eight; 128, in groups of 16, where there are more
// than 128, and from 65 on where logits have 16 bits and are kept so.  (262144 tokens, k =
// 8: 128 experts in bfloat16 59 us with 64 a thread, 53 with 128, 127 experts, read by 2
// bytes, 99 and 102; 128 in floats 62 and 81; 256 in bfloat16 111 and 87, in floats 113 and
// 102.  Fewer a thread leave room for more threads an SM, but each of a token's threads
// goes through every choice.)  With few tokens what counts is how long one takes: eight
// experts a thread.
struct Shape {
  int S, G;
  uint32_t lanes;
  uint64_t tiles;
};
Shape shape_of(uint32_t N, uint32_t E, bool narrow) {
  uint32_t eights = 1;  // groups of eight, a power of two
  while (eights * 8 < E) eights *= 2;
  Shape s = {8, (int)(eights < 8 ? eights : 8), eights <= 8 ? 1u : 2u, 0};
  const bool filled = N >= kForwardThreads * kSMs;  // a tile an SM, with a thread a token
  if (eights > 16 || (eights == 16 && narrow && filled)) s = {16, 8, eights / 16, 0};
  uint32_t tokens = kForwardThreads / s.lanes;
  s.tiles = ((uint64_t)N + tokens - 1) / tokens;
  if (s.tiles < kSMs) {
    s = {8, eights <= 32 ? 1 : (int)(eights / 32), eights <= 32 ? eights : 32, 0};
    tokens = kForwardThreads / s.lanes;
    s.tiles = ((uint64_t)N + tokens - 1) / tokens;
  }
  return s;
}

template <int S, int G, class T = float>
cudaError_t launch_forward(RouteParams &p, cudaStream_t st) {
  const size_t tokens = kForwardThreads / p.lanes, es = sizeof(T);
  size_t smem = 4 * (kForwardThreads * (size_t)(S * G * es / 4 + 4) + kForwardThreads * 4 / es +
                     p.lanes * S * G + 2 * tokens * p.k);
  smem = (smem + 15) / 16 * 16;  // the sums of a cluster's blocks start at a whole pair
  if (p.together) smem += 8 * (size_t)p.blocks * p.E;
  auto *k = route_forward_kernel<S, G, T>;
  cudaError_t e = allow_shared_memory((const void *)k);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.blocks);
  cfg.blockDim = dim3(kForwardThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.blocks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.together ? 1 : 0;
  ++launch_counter();
  e = cudaLaunchKernelEx(&cfg, k, (const RouteParams)p);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// A token's lanes backward, R experts each.
template <class E, int L, int R>
cudaError_t launch_backward(RouteParams &p, cudaStream_t st) {
  constexpr uint32_t kTokens = kWarps * (32 / L);  // a block takes at once
  const uint32_t blocks = (uint32_t)(((uint64_t)p.N + kTokens - 1) / kTokens);
  ++launch_counter();
  constexpr bool kNarrow = sizeof(E) == 2;
  const bool pairs = kNarrow && p.wide;
  auto *k = p.normalize ? pairs ? route_backward_kernel<E, L, R, kNarrow, true>
                                : route_backward_kernel<E, L, R, false, true>
            : pairs     ? route_backward_kernel<E, L, R, kNarrow, false>
                        : route_backward_kernel<E, L, R, false, false>;
  k<<<blocks < 8 * kSMs ? blocks : 8 * kSMs, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <class E>
cudaError_t backward_of(RouteParams &p, cudaStream_t st) {
  if (p.E <= 16) return launch_backward<E, 1, 16>(p, st);
  if (p.E <= 32) return launch_backward<E, 2, 16>(p, st);
  if (p.E <= 64) return launch_backward<E, 4, 16>(p, st);
  if (p.E <= 128) return launch_backward<E, 8, 16>(p, st);
  if (p.E <= 256) return launch_backward<E, 16, 16>(p, st);
  if (p.E <= 512) return launch_backward<E, 32, 16>(p, st);
  return launch_backward<E, 32, 32>(p, st);
}

RouteParams params_of(const ns_route_inputs &in) {
  RouteParams p = {};
  p.logits = in.logits, p.logits_row = in.logits_row, p.doc = in.doc, p.dtype = in.dtype;
  p.N = in.N, p.E = in.E, p.k = in.k, p.normalize = in.normalize != 0;
  return p;
}

// Bytes that rows can be moved by: 16, 8 or 4 where addresses, strides and widths
// are multiples of them, else 0.
int moved_at_once(const ns_route_inputs &in, const void *dlogits) {
  const uint64_t es = in.dtype == NS_F32 ? 4 : 2;
  const uint64_t all = (uint64_t)(uintptr_t)in.logits | (uint64_t)(uintptr_t)dlogits |
                       (uint64_t)in.logits_row * es | in.E * es;
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 0;
}

}  // namespace

static uint32_t blocks_of(uint64_t tiles) {
  // up to two tiles a block, one cluster does without the second kernel
  if (tiles <= 2 * kTogether) return 0;
  // as many blocks as an SM has room for: five (262144 tokens in bfloat16, k = 8: 64
  // experts 41 us with three, 38 with five; floats: 128 experts 69 and 58 us; 524288 tokens
  // of 8 experts, k = 2: 30 and 23 us)
  const uint32_t most = 5 * kSMs;
  return tiles < most ? (uint32_t)tiles : most;
}

uint32_t route_blocks(uint32_t N, uint32_t E) {  // of logits of either size
  return std::max(blocks_of(shape_of(N, E, false).tiles), blocks_of(shape_of(N, E, true).tiles));
}

cudaError_t launch_route_forward(const ns_route_inputs &in, int32_t *ids, float *weights,
                                 int32_t *counts, int32_t *tokens, float *loss, void *workspace,
                                 cudaStream_t st) {
  RouteParams p = params_of(in);
  const Shape shape = shape_of(in.N, in.E, in.dtype != NS_F32);
  p.wide = moved_at_once(in, nullptr), p.lanes = shape.lanes;
  p.ids = ids, p.weights = weights, p.counts = counts, p.tokens = tokens, p.loss = loss;
  p.blocks = blocks_of(shape.tiles);
  p.together = p.blocks == 0;
  if (p.together) p.blocks = shape.tiles < kTogether ? (uint32_t)shape.tiles : kTogether;
  if (p.blocks == 0) p.blocks = 1;  // no token: the counts are still written
  p.mass = static_cast<float *>(workspace);
  p.chosen = reinterpret_cast<int32_t *>(p.mass + (uint64_t)p.blocks * in.E);
  p.real = p.chosen + (uint64_t)p.blocks * in.E;
  const bool kept = shape.S == 16 && in.dtype != NS_F32;
  if (shape.S == 16 && !kept) p.blocks = std::min(p.blocks, 3 * kSMs);
  const cudaError_t e = kept ? in.dtype == NS_BF16 ? launch_forward<16, 8, __nv_bfloat16>(p, st)
                                                   : launch_forward<16, 8, __half>(p, st)
                        : shape.S == 16 ? launch_forward<16, 8>(p, st)
                        : shape.G == 8 ? launch_forward<8, 8>(p, st)
                        : shape.G == 4 ? launch_forward<8, 4>(p, st)
                        : shape.G == 2 ? launch_forward<8, 2>(p, st)
                                       : launch_forward<8, 1>(p, st);
  if (e != cudaSuccess || p.together) return e;
  ++launch_counter();
  pdl_launch(route_total_kernel, dim3(kFinalBlocks), dim3(kFinalThreads), 0, st, p);
  return cudaGetLastError();
}

cudaError_t launch_route_backward(const ns_route_inputs &in, const int32_t *ids,
                                  const float *weights, const int32_t *counts,
                                  const int32_t *tokens, const float *d_weights,
                                  const float *d_loss, void *dlogits, cudaStream_t st) {
  RouteParams p = params_of(in);
  p.ids = const_cast<int32_t *>(ids), p.weights = const_cast<float *>(weights);
  p.counts = const_cast<int32_t *>(counts), p.tokens = const_cast<int32_t *>(tokens);
  p.d_weights = d_weights, p.d_loss = d_loss, p.dlogits = dlogits;
  p.wide = moved_at_once(in, dlogits);
  switch (in.dtype) {
    case NS_F32: return backward_of<float>(p, st);
    case NS_BF16: return backward_of<__nv_bfloat16>(p, st);
    default: return backward_of<__half>(p, st);
  }
}

}  // namespace nsk
