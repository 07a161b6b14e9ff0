// Distillation from a teacher's top logits: the loss of every row and the
// gradient of its logits, in one pass over them.
//
//   q = softmax(s / temp) over V, p from the teacher's K entries, m = sum p
//   loss = temp^2 sum_k p_k (log p_k - log q_k),  ds_v = w temp (m q_v - p_v)
//
// The gradient needs the row's softmax sum before its first element can be
// written, and a row (256 KB for a vocabulary of 128K in 16 bits) is read from
// memory once: a cluster of C blocks keeps the row in its shared memory, a
// slice each, copied in with asynchronous 16-byte copies; every thread reduces
// the chunks that it copied itself to a running maximum and sum, the blocks
// exchange theirs through distributed shared memory, and each thread turns its
// chunks into the gradient.  The K entries of the teacher, which are few, are
// then written over what that put at their ids.
//
// Logits are kept as they came.  An exponential is 2^((s - max) log2 e / temp):
// the difference is taken first, so that it is exact where it matters, near the
// maximum, and a row at the type's lowest value does not overflow.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "train.h"

namespace nsk {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kGroups = 4;  // of asynchronous copies, waited for in order

struct DistillParams {
  const void *logits;
  int64_t logits_row;
  const void *top;
  const void *ids;
  const float *teacher_lse;
  const uint8_t *mask;
  const float *weight;
  uint32_t N, V, K;
  int32_t top_dtype, ids_64;
  float temp, inv_temp, scale;  // scale = log2 e / temp
  uint32_t slice;               // 16-byte chunks of a block's slice
  float *loss;
  void *dlogits;
  int64_t dlogits_row;
};

__device__ __forceinline__ void copy_wait_left(int left) {
  if (left == 3) copy_wait<3>();
  else if (left == 2) copy_wait<2>();
  else if (left == 1) copy_wait<1>();
  else copy_wait<0>();
}

// A running maximum (-inf at first) and the sum of exp((x - maximum) / temp).
struct MaxSum {
  float m, s;
};
// What is taken from x: the maximum, where -inf leaves x = -inf alone.
__device__ __forceinline__ float base_of(float m) { return m == kNegInf ? 0.0f : m; }
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float scale) {
  MaxSum r;
  r.m = fmaxf(a.m, b.m);
  const float base = base_of(r.m);
  r.s = a.s * exp2_sfu((a.m - base) * scale) + b.s * exp2_sfu((b.m - base) * scale);
  return r;
}

__device__ __forceinline__ float load_top(const void *top, int dtype, int64_t i) {
  if (dtype == NS_F32) return static_cast<const float *>(top)[i];
  if (dtype == NS_BF16) return to_f32(static_cast<const __nv_bfloat16 *>(top)[i]);
  return to_f32(static_cast<const __half *>(top)[i]);
}

// The row's K entries in shared memory, one array each.
struct Entries {
  int *id;      // -1: absent
  float *p;     // probability
  float *logp;  // its natural logarithm
  float *x;     // the student's logit there, where this block holds it
};

// Warp 0: the teacher's probabilities; returns their sum m (1 unless the
// teacher's own normaliser is given, 0 if no entry is left).
__device__ float teacher_entries(const DistillParams &p, uint32_t row, int lane,
                                 const Entries &e) {
  const int64_t base = (int64_t)row * p.K;
  float m = kNegInf;
  for (uint32_t k = lane; k < p.K; k += 32) {
    const int64_t id = p.ids_64 ? static_cast<const int64_t *>(p.ids)[base + k]
                                : (int64_t)static_cast<const int32_t *>(p.ids)[base + k];
    const float t = load_top(p.top, p.top_dtype, base + k);
    const bool in = id >= 0 && id < (int64_t)p.V;
    e.id[k] = in ? (int)id : -1;
    e.logp[k] = in ? t : kNegInf;
    if (in) m = fmaxf(m, t);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base_m = base_of(m);
  const float lse = p.teacher_lse ? p.teacher_lse[row] : 0.0f;
  float sum = 0.0f;
  for (uint32_t k = lane; k < p.K; k += 32) {
    const float t = e.logp[k];
    const float l = p.teacher_lse ? fmaf(t, p.inv_temp, -lse) : (t - base_m) * p.inv_temp;
    // an absent entry stays at -inf whatever lse is
    const float keep = e.id[k] < 0 ? kNegInf : l;
    const float v = expf(keep);
    e.logp[k] = keep;
    e.p[k] = v;
    sum += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (p.teacher_lse) return sum;
  if (sum == 0.0f) return 0.0f;
  const float inv = 1.0f / sum, log_sum = logf(sum);
  for (uint32_t k = lane; k < p.K; k += 32) {
    e.p[k] *= inv;
    e.logp[k] -= log_sum;
  }
  return 1.0f;
}

template <class E, bool kGrad>
__global__ void __launch_bounds__(kMaxThreads) distill_kernel(const DistillParams p) {
  constexpr int kN = 16 / sizeof(E);  // elements of a chunk
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 stats[kMaxCluster];   // (maximum, sum) of every block's slice
  __shared__ float losses[kMaxCluster];   // in block 0: every block's part of the loss
  __shared__ float2 warp_stats[kMaxThreads / 32];
  __shared__ float warp_loss[kMaxThreads / 32];
  __shared__ float mass;
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const uint32_t row = blockIdx.x / C;
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;

  // The row in chunks of 16 bytes from the boundary at or below its start.
  const E *src = static_cast<const E *>(p.logits) + (int64_t)row * p.logits_row;
  const int mis = (int)(((uintptr_t)src & 15) / sizeof(E));
  const uint32_t chunks = (uint32_t)(((uint64_t)mis + p.V + kN - 1) / kN);
  const uint32_t first = min(rank * p.slice, chunks), mine = min(p.slice, chunks - first);
  const int64_t e0 = (int64_t)first * kN - mis;  // index of this slice's first element
  E *dst = kGrad ? static_cast<E *>(p.dlogits) + (int64_t)row * p.dlogits_row : nullptr;
  // whole chunks of the gradient can be stored at once
  const bool wide = kGrad && ((uintptr_t)(dst - mis) & 15) == 0;
  auto store_chunk = [&](uint32_t c, const Vec<E, kN> &v) {
    const int64_t i = e0 + (int64_t)c * kN;
    if (wide && i >= 0 && i + kN <= (int64_t)p.V) {
      *reinterpret_cast<Vec<E, kN> *>(dst + i) = v;
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k)
        if (i + k >= 0 && i + k < (int64_t)p.V) dst[i + k] = v.v[k];
    }
  };

  if (p.mask && p.mask[row] == 0) {  // the same for every block of the cluster
    if (kGrad) {
      Vec<E, kN> zero;
#pragma unroll
      for (int k = 0; k < kN; ++k) zero.v[k] = from_f32<E>(0.0f);
      for (uint32_t c = tid; c < mine; c += nthr) store_chunk(c, zero);
    }
    if (rank == 0 && tid == 0) p.loss[row] = 0.0f;
    return;
  }
  cluster_arrive();  // waited for before the first write to another block

  // Copies of this thread's chunks, in kGroups groups.
  E *slice = reinterpret_cast<E *>(smem);
  const uint32_t per = (mine + nthr - 1) / nthr;  // chunks of a thread
  uint32_t j = 0;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint32_t end = (per * (g + 1) + kGroups - 1) / kGroups;
    for (; j < end; ++j) {
      const uint32_t c = j * nthr + tid;
      if (c < mine) {
        const int64_t i = e0 + (int64_t)c * kN;
        if (i >= 0 && i + kN <= (int64_t)p.V) {
          copy_async<16>(slice + (size_t)c * kN, src + i);
        } else {  // the row's ends
#pragma unroll
          for (int k = 0; k < kN; ++k)
            slice[(size_t)c * kN + k] = i + k >= 0 && i + k < (int64_t)p.V
                                            ? src[i + k]
                                            : from_f32<E>(kNegInf);
        }
      }
    }
    copy_commit();
  }

  Entries e;
  e.p = reinterpret_cast<float *>(smem + (size_t)p.slice * 16);
  e.logp = e.p + p.K;
  e.x = e.logp + p.K;
  e.id = reinterpret_cast<int *>(e.x + p.K);
  if (warp == 0) {
    const float m = teacher_entries(p, row, lane, e);
    if (lane == 0) mass = m;
  }

  // Maximum and sum of this thread's chunks, as they arrive.
  MaxSum acc = {kNegInf, 0.0f};
  j = 0;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint32_t end = (per * (g + 1) + kGroups - 1) / kGroups;
    copy_wait_left(kGroups - 1 - g);
    for (; j < end; ++j) {
      const uint32_t c = j * nthr + tid;
      if (c < mine) {
        const Vec<E, kN> v = *reinterpret_cast<const Vec<E, kN> *>(slice + (size_t)c * kN);
        float x[kN], top = to_f32(v.v[0]);
#pragma unroll
        for (int k = 0; k < kN; ++k) x[k] = to_f32(v.v[k]);
#pragma unroll
        for (int k = 1; k < kN; ++k) top = fmaxf(top, x[k]);
        if (top > acc.m) {
          acc.s *= exp2_sfu((acc.m - top) * p.scale);
          acc.m = top;
        }
        const float base = base_of(acc.m);
#pragma unroll
        for (int k = 0; k < kN; ++k) acc.s += exp2_sfu((x[k] - base) * p.scale);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const MaxSum other = {__shfl_xor_sync(0xffffffffu, acc.m, o),
                          __shfl_xor_sync(0xffffffffu, acc.s, o)};
    acc = join(acc, other, p.scale);
  }
  if (lane == 0) warp_stats[warp] = make_float2(acc.m, acc.s);
  __syncthreads();  // also: the slice and the entries are in shared memory
  cluster_wait();   // every block of the cluster has started
  if (tid < (int)C) {
    acc = {warp_stats[0].x, warp_stats[0].y};
    for (int w = 1; w < nthr / 32; ++w)
      acc = join(acc, {warp_stats[w].x, warp_stats[w].y}, p.scale);
    remote_store(remote_smem(&stats[rank], tid), make_float2(acc.m, acc.s));
  }
  cluster_arrive();
  cluster_wait();
  acc = {stats[0].x, stats[0].y};
  for (uint32_t r = 1; r < C; ++r) acc = join(acc, {stats[r].x, stats[r].y}, p.scale);
  const float base = base_of(acc.m), m = mass;
  const float log_s = logf(acc.s);

  // The entries whose ids lie in this slice: their student logits, and their
  // part of the loss.
  float part = 0.0f;
  for (uint32_t k = tid; k < p.K; k += nthr) {
    const int64_t at = (int64_t)e.id[k] - e0;
    if (e.id[k] >= 0 && at >= 0 && at < (int64_t)mine * kN) {
      const float x = to_f32(slice[at]), pk = e.p[k];
      e.x[k] = x;
      const float log_q = x == kNegInf ? kNegInf : fmaf(x - base, p.inv_temp, -log_s);
      if (pk != 0.0f) part += pk * (e.logp[k] - log_q);
    } else {
      e.id[k] = -1;  // another block's, or absent
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) warp_loss[warp] = part;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < nthr / 32; ++w) part += warp_loss[w];
    remote_store(remote_smem(&losses[rank], 0), part);
  }
  cluster_arrive();

  if (kGrad) {
    const float w = (p.weight ? p.weight[row] : 1.0f) * p.temp;
    const float f = m == 0.0f || acc.s == 0.0f ? 0.0f : w * m / acc.s;  // of the exponentials
    const bool none = m == 0.0f;
    for (uint32_t c = tid; c < mine; c += nthr) {
      const Vec<E, kN> v = *reinterpret_cast<const Vec<E, kN> *>(slice + (size_t)c * kN);
      Vec<E, kN> out;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const float g = f * exp2_sfu((to_f32(v.v[k]) - base) * p.scale);
        out.v[k] = from_f32<E>(none ? 0.0f : g);
      }
      store_chunk(c, out);
    }
    __syncthreads();  // the slice is read, the gradient is written
    // Of entries with the same id, one writes the sum of their p: the one
    // whose number is left in the slice at that id.
    using Tag = typename std::conditional<sizeof(E) == 2, uint16_t, uint32_t>::type;
    Tag *tags = reinterpret_cast<Tag *>(smem);
    for (uint32_t k = tid; k < p.K; k += nthr)
      if (e.id[k] >= 0) tags[e.id[k] - e0] = (Tag)k;
    __syncthreads();
    bool twice = false;
    for (uint32_t k = tid; k < p.K; k += nthr)
      if (e.id[k] >= 0 && tags[e.id[k] - e0] != (Tag)k) twice = true;
    twice = __syncthreads_or(twice);
    for (uint32_t k = tid; k < p.K; k += nthr) {
      if (e.id[k] < 0 || tags[e.id[k] - e0] != (Tag)k) continue;
      float pk = e.p[k];
      if (twice) {  // in the entries' order
        pk = 0.0f;
        for (uint32_t i = 0; i < p.K; ++i)
          if (e.id[i] == e.id[k]) pk += e.p[i];
      }
      const float g = f * exp2_sfu((e.x[k] - base) * p.scale);
      dst[e.id[k]] = from_f32<E>(none ? 0.0f : fmaf(-w, pk, g));
    }
  }
  cluster_wait();  // every block's part of the loss is in block 0
  if (rank == 0 && tid == 0) {
    float loss = losses[0];
    for (uint32_t r = 1; r < C; ++r) loss += losses[r];
    p.loss[row] = loss * p.temp * p.temp;
  }
}

// Bytes of shared memory of a block's slice that let three blocks share an SM.
constexpr uint64_t kSliceBytes = 66 * 1024;

template <class E, bool kGrad>
cudaError_t launch(DistillParams &p, cudaStream_t st) {
  // chunks of a row at its least favourable alignment
  const uint64_t bytes = ((uint64_t)p.V * sizeof(E) + 15 + 15) / 16 * 16;
  uint32_t C = 1;
  while (C < kMaxCluster && bytes > C * kSliceBytes) C *= 2;
  p.slice = (uint32_t)((bytes / 16 + C - 1) / C);
  const size_t smem = (size_t)p.slice * 16 + (size_t)p.K * 16;
  const unsigned threads = p.slice >= 2048 ? 512 : p.slice >= 512 ? 256 : 128;
  auto *k = distill_kernel<E, kGrad>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.N * C);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  ++launch_counter();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, (const DistillParams)p);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

}  // namespace

cudaError_t launch_distill(const ns_distill_inputs &in, float *loss, void *dlogits,
                           int64_t dlogits_row, cudaStream_t st) {
  DistillParams p = {};
  p.logits = in.logits, p.logits_row = in.logits_row;
  p.top = in.top_logits, p.ids = in.top_ids, p.teacher_lse = in.teacher_lse;
  p.mask = in.mask, p.weight = in.weight;
  p.N = in.N, p.V = in.V, p.K = in.K;
  p.top_dtype = in.top_dtype, p.ids_64 = in.ids_64;
  p.temp = in.temperature, p.inv_temp = 1.0f / in.temperature;
  p.scale = (float)(1.4426950408889634 / in.temperature);
  p.loss = loss, p.dlogits = dlogits, p.dlogits_row = dlogits_row;
  switch (in.dtype) {
    case NS_F32: return dlogits ? launch<float, true>(p, st) : launch<float, false>(p, st);
    case NS_BF16:
      return dlogits ? launch<__nv_bfloat16, true>(p, st) : launch<__nv_bfloat16, false>(p, st);
    default: return dlogits ? launch<__half, true>(p, st) : launch<__half, false>(p, st);
  }
}

}  // namespace nsk
