// A router over packed positions: softmax over E logits a token, its k largest,
// per-expert counts, the balance loss, and the logits' gradient.
//
//   loss = E / (k M^2) sum_e counts_e mass_e,  mass_e = sum_n p_ne
//   dl_nj = p_nj (g_j - sum_e p_ne g_e) + the chosen weights' part,
//   g_e = d_loss E / (k M^2) counts_e
//
// L lanes of a warp take a token, R consecutive experts each, all in
// registers: one read of the logits, shuffles of log2 L steps for the row's
// maximum and sum and for each of the k choices.  A choice is the maximum of
// keys that order the logits and, of equal ones, put the lowest index first.
// Each lane adds its experts' probabilities up over all of its tokens; blocks
// write rows of partial sums and counts, and a second kernel adds them in a
// fixed order (no floating-point atomics: the loss has the same bits every
// time).  The backward pass reads the logits again and computes the softmax
// again, which costs less than keeping it.
#include <cuda_runtime.h>

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
constexpr uint32_t kMaxBlocks = 456;  // three blocks on each of 152 SMs

struct RouteParams {
  const void *logits;
  int64_t logits_row;
  const int32_t *doc;
  uint32_t N, E, k;
  int32_t normalize, wide;  // wide: a lane's experts can be moved at once
  int32_t *ids;
  float *weights;
  // forward
  float *mass;      // [blocks][E]
  int32_t *chosen;  // [blocks][E]
  int32_t *real;    // [blocks]
  int32_t *counts, *tokens;
  float *loss;
  uint32_t blocks;
  // backward
  const float *d_weights, *d_loss;
  void *dlogits;
};

// Keys: unsigned numbers in the order of (logit, then lowest index first), 0
// for an expert that cannot be chosen (-inf, NaN).  A 16-bit type's value and the index
// fit 32 bits together; a float needs 64.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 and 0 are equal
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
template <class E>
struct KeyOf {
  using type = uint32_t;
  // bits below the value's: bfloat16 has 16 significant ones as a float, half 19
  static constexpr uint32_t kLow = sizeof(E) == 4 ? 0u
                                   : std::is_same<E, __half>::value ? 0x1fffu : 0xffffu;
  static __device__ __forceinline__ uint32_t make(float x, uint32_t i) {
    return (ordered(x) & ~kLow) | (kLow - i);
  }
  static __device__ __forceinline__ uint32_t index(uint32_t key) { return kLow - (key & kLow); }
  static __device__ __forceinline__ float value(uint32_t key) {
    const uint32_t hi = key & ~kLow;
    return unordered(hi & 0x80000000u ? hi : hi | kLow);
  }
};
template <>
struct KeyOf<float> {
  using type = uint64_t;
  static __device__ __forceinline__ uint64_t make(float x, uint32_t i) {
    return (uint64_t)ordered(x) << 32 | (0xffffffffu - i);
  }
  static __device__ __forceinline__ uint32_t index(uint64_t key) {
    return 0xffffffffu - (uint32_t)key;
  }
  static __device__ __forceinline__ float value(uint64_t key) {
    return unordered((uint32_t)(key >> 32));
  }
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
template <int L>
__device__ __forceinline__ uint64_t group_best(uint64_t v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = w > v ? w : v;
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_best(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}

// Elements of one access of at most 16 bytes.
template <class E, int R>
constexpr int kMove = R * sizeof(E) <= 16 ? R : 16 / sizeof(E);

// The lane's experts of token n (-inf where there is none or `real` is false).
template <class E, int R>
__device__ __forceinline__ void load_logits(const RouteParams &p, uint32_t n, uint32_t i0,
                                            bool real, float (&x)[R]) {
  constexpr int kN = kMove<E, R>;
#pragma unroll
  for (int r = 0; r < R; ++r) x[r] = kNegInf;
  if (!real) return;
  const E *src = static_cast<const E *>(p.logits) + (int64_t)n * p.logits_row + i0;
  if (p.wide) {
    if (i0 < p.E) {
#pragma unroll
      for (int r = 0; r < R; r += kN) {
        const Vec<E, kN> v = *reinterpret_cast<const Vec<E, kN> *>(src + r);
#pragma unroll
        for (int q = 0; q < kN; ++q) x[r + q] = to_f32(v.v[q]);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i0 + r < p.E) x[r] = to_f32(src[r]);
  }
}

// Softmax of a token: x becomes exp(x - max), and their sum is returned (0 for
// a token that counts for nothing).  The difference is taken before the change
// of base, which overflows for logits near the type's lowest value.
template <int L, int R>
__device__ __forceinline__ float exponentials(float (&x)[R], float &base) {
  float m = x[0];
#pragma unroll
  for (int r = 1; r < R; ++r) m = fmaxf(m, x[r]);
  m = group_max<L>(m);
  base = m == kNegInf ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    x[r] = exp2_sfu((x[r] - base) * kLog2e);
    s += x[r];
  }
  return group_sum<L>(s);
}

__device__ __forceinline__ float balance(uint32_t E, uint32_t k, int32_t M) {
  return M == 0 ? 0.0f : (float)E / (float)k / ((float)M * (float)M);
}

template <class E, int L, int R>
__global__ void __launch_bounds__(kThreads) route_forward_kernel(const RouteParams p) {
  using Key = typename KeyOf<E>::type;
  constexpr int G = 32 / L, kExperts = L * R, kTop = kExperts < 32 ? kExperts : 32;
  __shared__ float mass[kWarps][kExperts];
  __shared__ int chosen[kExperts];
  __shared__ int top_id[kWarps][G][kTop];
  __shared__ float top_e[kWarps][G][kTop];
  __shared__ int real_tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / L, gl = lane % L;
  const uint32_t i0 = gl * R;
  for (int e = threadIdx.x; e < kExperts; e += kThreads) chosen[e] = 0;
  if (threadIdx.x == 0) real_tokens = 0;
  __syncthreads();
  float sum[R];
#pragma unroll
  for (int r = 0; r < R; ++r) sum[r] = 0.0f;
  int counted = 0;
  int *my_id = top_id[warp][group];
  float *my_e = top_e[warp][group];
  const uint64_t step = (uint64_t)gridDim.x * kWarps * G;
  for (uint64_t n0 = ((uint64_t)blockIdx.x * kWarps + warp) * G; n0 < p.N; n0 += step) {
    const bool in = n0 + group < p.N;
    const uint32_t n = in ? (uint32_t)(n0 + group) : 0;
    const bool real = in && !(p.doc && __ldg(p.doc + n) < 0);
    float x[R], base;
    load_logits<E, R>(p, n, i0, real, x);
    Key key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) key[r] = x[r] > kNegInf ? KeyOf<E>::make(x[r], i0 + r) : 0;
    const float s = exponentials<L, R>(x, base);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int r = 0; r < R; ++r) sum[r] += s == 0.0f ? 0.0f : x[r] * inv;
    if (gl == 0 && s != 0.0f) ++counted;
    for (uint32_t j = 0; j < p.k; ++j) {
      Key best = key[0];
#pragma unroll
      for (int r = 1; r < R; ++r) best = key[r] > best ? key[r] : best;
      best = group_best<L>(best);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (key[r] == best) key[r] = 0;
      if (gl == 0) {
        my_id[j] = best == 0 ? -1 : (int)KeyOf<E>::index(best);
        my_e[j] = best == 0 ? 0.0f : exp2_sfu((KeyOf<E>::value(best) - base) * kLog2e);
      }
    }
    __syncwarp();
    float total = 0.0f;
    if (p.normalize) {
      for (uint32_t j = gl; j < p.k; j += L) total += my_e[j];
      total = group_sum<L>(total);
    }
    // a NaN logit is never chosen, but makes s and so the token's weights NaN
    const float by = p.normalize ? (total == 0.0f ? 0.0f : 1.0f / total) + (s - s) : inv;
    for (uint32_t j = gl; in && j < p.k; j += L) {
      const int id = my_id[j];
      p.ids[(int64_t)n * p.k + j] = id;
      p.weights[(int64_t)n * p.k + j] = id < 0 ? 0.0f : my_e[j] * by;
      if (id >= 0) atomicAdd(&chosen[id], 1);
    }
    __syncwarp();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
    if (group == 0) mass[warp][i0 + r] = sum[r];
  }
  counted = warp_sum_i32(counted);
  if (lane == 0) atomicAdd(&real_tokens, counted);
  __syncthreads();
  float part = 0.0f;
  for (uint32_t e = threadIdx.x; e < p.E; e += kThreads) {
    float v = mass[0][e];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += mass[w][e];
    if (p.blocks == 1) {
      p.counts[e] = chosen[e];
      part += v * (float)chosen[e];
    } else {
      p.mass[(uint64_t)blockIdx.x * p.E + e] = v;
      p.chosen[(uint64_t)blockIdx.x * p.E + e] = chosen[e];
    }
  }
  if (p.blocks == 1) {  // few tokens: this block has all of them
    part = group_sum<32>(part);
    __syncthreads();
    if (lane == 0) mass[warp][0] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) part += mass[w][0];
      p.tokens[0] = real_tokens;
      p.loss[0] = part * balance(p.E, p.k, real_tokens);
    }
  } else if (threadIdx.x == 0) {
    p.real[blockIdx.x] = real_tokens;
  }
}

// The blocks' partial sums, added up by one cluster: block c of it takes a
// share of the experts, `width` lanes side by side and the rest of its threads
// down the rows.
constexpr int kFinalThreads = 512;
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
#pragma unroll 4
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

template <class E, int L, int R>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteParams p) {
  constexpr int G = 32 / L, kExperts = L * R;
  __shared__ __align__(16) float add[kWarps][G][kExperts];  // the weights' part, 0 elsewhere
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / L, gl = lane % L;
  const uint32_t i0 = gl * R;
  float *my_add = add[warp][group];
  float g[R];
  const float coef =
      p.d_loss ? p.d_loss[0] * balance(p.E, p.k, p.tokens[0]) : 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    g[r] = p.d_loss && i0 + r < p.E ? coef * (float)p.counts[i0 + r] : 0.0f;
    my_add[i0 + r] = 0.0f;
  }
  __syncwarp();
  const uint64_t step = (uint64_t)gridDim.x * kWarps * G;
  for (uint64_t n0 = ((uint64_t)blockIdx.x * kWarps + warp) * G; n0 < p.N; n0 += step) {
    const bool in = n0 + group < p.N;
    const uint32_t n = in ? (uint32_t)(n0 + group) : 0;
    const bool real = in && !(p.doc && __ldg(p.doc + n) < 0);
    float x[R], base;
    load_logits<E, R>(p, n, i0, real, x);
    const float s = exponentials<L, R>(x, base);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    float dot = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] *= inv;
      dot += x[r] * g[r];
    }
    dot = group_sum<L>(dot);
    if (p.d_weights) {
      // w = p at the chosen ones: dl_j = w_j dw_j - p_j t at them, t = sum w dw;
      // normalised, w is their own softmax: dl_j = w_j (dw_j - t)
      float t = 0.0f;
      for (uint32_t j = gl; real && j < p.k; j += L)
        if (p.ids[(int64_t)n * p.k + j] >= 0)  // else there is no such choice
          t += p.weights[(int64_t)n * p.k + j] * p.d_weights[(int64_t)n * p.k + j];
      t = group_sum<L>(t);
      for (uint32_t j = gl; real && j < p.k; j += L) {
        const int id = p.ids[(int64_t)n * p.k + j];
        const float w = p.weights[(int64_t)n * p.k + j];
        if (id >= 0 && id < (int)p.E)
          my_add[id] = w * (p.d_weights[(int64_t)n * p.k + j] - (p.normalize ? t : 0.0f));
      }
      if (!p.normalize) dot += t;
      __syncwarp();
    }
    if (in) {
      constexpr int kN = kMove<E, R>;
      E *dst = static_cast<E *>(p.dlogits) + (int64_t)n * p.E + i0;
      float d[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        d[r] = x[r] * (g[r] - dot);
        if (p.d_weights) d[r] += my_add[i0 + r];
        if (s == 0.0f) d[r] = 0.0f;
      }
      if (p.wide) {
        if (i0 < p.E) {
#pragma unroll
          for (int r = 0; r < R; r += kN) {
            Vec<E, kN> v;
#pragma unroll
            for (int q = 0; q < kN; ++q) v.v[q] = from_f32<E>(d[r + q]);
            *reinterpret_cast<Vec<E, kN> *>(dst + r) = v;
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (i0 + r < p.E) dst[r] = from_f32<E>(d[r]);
      }
    }
    if (p.d_weights) {
      __syncwarp();
      for (uint32_t j = gl; real && j < p.k; j += L) {
        const int id = p.ids[(int64_t)n * p.k + j];
        if (id >= 0 && id < (int)p.E) my_add[id] = 0.0f;
      }
      __syncwarp();
    }
  }
}

// Lanes of a token: as many as hold its experts, eight each.
int lanes_of(uint32_t E) {
  int L = 2;
  while (L < 32 && (uint32_t)L * 8 < E) L *= 2;
  return L;
}

template <class E, int L, int R, bool kForward>
cudaError_t launch(RouteParams &p, uint32_t blocks, cudaStream_t st) {
  ++launch_counter();
  if (kForward)
    route_forward_kernel<E, L, R><<<blocks, kThreads, 0, st>>>(p);
  else
    route_backward_kernel<E, L, R><<<blocks, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <class E, bool kForward>
cudaError_t by_experts(RouteParams &p, uint32_t blocks, cudaStream_t st) {
  if (p.E <= 16) return launch<E, 2, 8, kForward>(p, blocks, st);
  if (p.E <= 32) return launch<E, 4, 8, kForward>(p, blocks, st);
  if (p.E <= 64) return launch<E, 8, 8, kForward>(p, blocks, st);
  if (p.E <= 128) return launch<E, 16, 8, kForward>(p, blocks, st);
  if (p.E <= 256) return launch<E, 32, 8, kForward>(p, blocks, st);
  if (p.E <= 512) return launch<E, 32, 16, kForward>(p, blocks, st);
  return launch<E, 32, 32, kForward>(p, blocks, st);
}

template <bool kForward>
cudaError_t by_type(RouteParams &p, int dtype, uint32_t blocks, cudaStream_t st) {
  const size_t es = dtype == NS_F32 ? 4 : 2;
  const uint32_t R = p.E <= 256 ? 8 : p.E <= 512 ? 16 : 32;
  p.wide = p.E % R == 0 && (uintptr_t)p.logits % 16 == 0 && (p.logits_row * es) % 16 == 0 &&
           (uintptr_t)p.dlogits % 16 == 0;
  switch (dtype) {
    case NS_F32: return by_experts<float, kForward>(p, blocks, st);
    case NS_BF16: return by_experts<__nv_bfloat16, kForward>(p, blocks, st);
    default: return by_experts<__half, kForward>(p, blocks, st);
  }
}

RouteParams params_of(const ns_route_inputs &in) {
  RouteParams p = {};
  p.logits = in.logits, p.logits_row = in.logits_row, p.doc = in.doc;
  p.N = in.N, p.E = in.E, p.k = in.k, p.normalize = in.normalize != 0;
  return p;
}

}  // namespace

uint32_t route_blocks(uint32_t N, uint32_t E) {
  const uint32_t per = kWarps * (32 / lanes_of(E));  // tokens a block takes at once
  const uint64_t blocks = ((uint64_t)N + per - 1) / per;
  // up to four rounds of one block are quicker than a second kernel
  return blocks <= 4 ? 1 : blocks < kMaxBlocks ? (uint32_t)blocks : kMaxBlocks;
}

cudaError_t launch_route_forward(const ns_route_inputs &in, int32_t *ids, float *weights,
                                 int32_t *counts, int32_t *tokens, float *loss, void *workspace,
                                 cudaStream_t st) {
  RouteParams p = params_of(in);
  p.ids = ids, p.weights = weights, p.counts = counts, p.tokens = tokens, p.loss = loss;
  p.blocks = route_blocks(in.N, in.E);
  p.mass = static_cast<float *>(workspace);
  p.chosen = reinterpret_cast<int32_t *>(p.mass + (uint64_t)p.blocks * in.E);
  p.real = p.chosen + (uint64_t)p.blocks * in.E;
  const cudaError_t e = by_type<true>(p, in.dtype, p.blocks, st);
  if (e != cudaSuccess || p.blocks == 1) return e;
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
  const uint32_t per = kWarps * (32 / lanes_of(in.E));
  const uint64_t blocks = ((uint64_t)in.N + per - 1) / per;
  return by_type<false>(p, in.dtype, blocks < 4 * kMaxBlocks ? (uint32_t)blocks : 4 * kMaxBlocks,
                        st);
}

}  // namespace nsk
