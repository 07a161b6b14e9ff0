// Distillation from a teacher's top logits: the loss of every row and the
// gradient of its logits, in one pass over them.
//
//   q = softmax(s / temp) over V, p from the teacher's K entries, m = sum p
//   loss = temp^2 sum_k p_k (log p_k - log q_k),  ds_v = w temp (m q_v - p_v)
//
// The gradient needs the row's softmax sum before its first element can be
// written, and a row (256 KB for a vocabulary of 128K in 16 bits) is read from
// memory once: a cluster of C blocks keeps the row in its shared memory, a slice
// each, copied in with asynchronous 16-byte copies; every thread reduces the chunks
// that it copied itself to a running maximum and sum, the blocks exchange theirs
// through distributed shared memory, and each thread turns its chunks into the
// gradient.  The teacher's K entries are few: one warp of each block has them.  It
// adds up the loss of those whose ids lie in its slice before the exchange, so that
// one is enough:
//   sum_k p_k (log p_k - log q_k) = sum over the slices r of
//     part_r + pm_r (log S + (M - m_r) / temp),
//   part_r = sum of p_k (log p_k - (s_k - m_r) / temp), pm_r = sum of p_k there,
// with M, S the row's maximum and sum and m_r the slice's maximum (which keeps the
// terms small).  After the gradient is written it writes the entries' own over it.
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
  int *id;      // -1: absent, or (later) in another block's slice
  float *p;     // probability
  float *logp;  // its natural logarithm
  float *x;     // the student's logit there
};

// What an entry's number is kept in, over a logit.
template <class E>
using Tag = typename std::conditional<sizeof(E) == 2, uint16_t, uint32_t>::type;

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
__global__ void __launch_bounds__(kMaxThreads, 3) distill_kernel(const DistillParams p) {
  constexpr int kN = 16 / sizeof(E);  // elements of a chunk
  extern __shared__ __align__(16) unsigned char smem[];
  // every slice's maximum, sum, part_r and pm_r
  __shared__ __align__(16) float4 stats[kMaxCluster];
  __shared__ float2 warp_stats[kMaxThreads / 32];
  __shared__ float mass_of_row;
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const uint32_t row = blockIdx.x / C;
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;

  // The row in chunks of 16 bytes from the boundary at or below its start.
  const E *src = static_cast<const E *>(p.logits) + (int64_t)row * p.logits_row;
  const int mis = (int)(((uintptr_t)src & 15) / sizeof(E));
  const uint32_t chunks = (uint32_t)(((uint64_t)mis + p.V + kN - 1) / kN);
  const uint32_t first = min(rank * p.slice, chunks), mine = min(p.slice, chunks - first);
  const int e0 = (int)(first * kN) - mis;  // index of this slice's first element
  // chunks [whole, whole + wholes) lie inside the row, at most one on either side does not
  const uint32_t whole = e0 < 0 ? 1 : 0;
  const uint32_t wholes =
      mine - whole - (mine > whole && e0 + (int)mine * kN > (int)p.V ? 1 : 0);
  E *dst = kGrad ? static_cast<E *>(p.dlogits) + (int64_t)row * p.dlogits_row : nullptr;
  // whole chunks of the gradient can be stored at once
  const bool wide = kGrad && ((uintptr_t)(dst - mis) & 15) == 0;
  auto store_chunk = [&](uint32_t c, uint4 v) {
    E *to = dst + e0 + (int)(c * kN);
    if (wide && c - whole < wholes) {
      *reinterpret_cast<uint4 *>(to) = v;
    } else {
      E x[kN];
      *reinterpret_cast<uint4 *>(x) = v;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int i = e0 + (int)(c * kN) + k;
        if (i >= 0 && i < (int)p.V) to[k] = x[k];
      }
    }
  };

  if (p.mask && p.mask[row] == 0) {  // the same for every block of the cluster
    if (kGrad)
      for (uint32_t c = tid; c < mine; c += nthr) store_chunk(c, make_uint4(0, 0, 0, 0));
    if (rank == 0 && tid == 0) p.loss[row] = 0.0f;
    return;
  }
  cluster_arrive_relaxed();  // waited for before the first write to another block

  // Copies of this thread's chunks, in kGroups groups.
  uint4 *slice = reinterpret_cast<uint4 *>(smem);
  const uint32_t per = (mine + nthr - 1) / nthr;  // chunks of a thread
  uint32_t c = tid;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint32_t end = min((per * (g + 1) + kGroups - 1) / kGroups * nthr, mine);
    for (; c < end; c += nthr) {
      const E *from = src + e0 + (int)(c * kN);
      if (c - whole < wholes) {
        copy_async<16>(slice + c, from);
      } else {  // the row's ends
        E x[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const int i = e0 + (int)(c * kN) + k;
          x[k] = i >= 0 && i < (int)p.V ? from[k] : from_f32<E>(kNegInf);
        }
        slice[c] = *reinterpret_cast<const uint4 *>(x);
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
    if (lane == 0) mass_of_row = m;
  }

  // Maximum and sum of this thread's chunks, as they arrive.
  MaxSum acc = {kNegInf, 0.0f};
  const Ch<2> scale = splat<2>(p.scale);
  c = tid;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint32_t end = min((per * (g + 1) + kGroups - 1) / kGroups * nthr, mine);
    copy_wait_left(kGroups - 1 - g);
#pragma unroll 2
    for (; c < end; c += nthr) {
      Ch<2> x[kN / 2];
      widen_chunk<E>(slice[c], x);
      float top = fmaxf(x[0].v[0], x[0].v[1]);
#pragma unroll
      for (int k = 1; k < kN / 2; ++k) top = fmaxf(top, fmaxf(x[k].v[0], x[k].v[1]));
      if (top > acc.m) {
        acc.s *= exp2_sfu((acc.m - top) * p.scale);
        acc.m = top;
      }
      const Ch<2> base = splat<2>(-base_of(acc.m));
      Ch<2> sum;
#pragma unroll
      for (int k = 0; k < kN / 2; ++k) {
        const Ch<2> y = (x[k] + base) * scale;
        const Ch<2> v = {exp2_sfu(y.v[0]), exp2_sfu(y.v[1])};
        sum = k == 0 ? v : sum + v;
      }
      acc.s += sum.v[0] + sum.v[1];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const MaxSum other = {__shfl_xor_sync(0xffffffffu, acc.m, o),
                          __shfl_xor_sync(0xffffffffu, acc.s, o)};
    acc = join(acc, other, p.scale);
  }
  if (lane == 0) warp_stats[warp] = make_float2(acc.m, acc.s);
  __syncthreads();  // also: the slice is in shared memory
  if (warp == 0) {
    acc = {kNegInf, 0.0f};
    if (lane < nthr / 32) acc = {warp_stats[lane].x, warp_stats[lane].y};
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const MaxSum other = {__shfl_xor_sync(0xffffffffu, acc.m, o),
                            __shfl_xor_sync(0xffffffffu, acc.s, o)};
      acc = join(acc, other, p.scale);
    }
    // lanes 16 and up joined nothing: lane 0 has the slice's
    acc = {__shfl_sync(0xffffffffu, acc.m, 0), __shfl_sync(0xffffffffu, acc.s, 0)};
    const float base = base_of(acc.m);
    float part = 0.0f, pm = 0.0f;
    for (uint32_t k = lane; k < p.K; k += 32) {
      const int at = e.id[k] - e0;
      if (e.id[k] >= 0 && at >= 0 && at < (int)(mine * kN)) {
        const float x = to_f32(reinterpret_cast<const E *>(slice)[at]), pk = e.p[k];
        e.x[k] = x;
        if (pk != 0.0f) {
          part += pk * (x == kNegInf ? -kNegInf : fmaf(base - x, p.inv_temp, e.logp[k]));
          pm += pk;
        }
      } else {
        e.id[k] = -1;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      part += __shfl_xor_sync(0xffffffffu, part, o);
      pm += __shfl_xor_sync(0xffffffffu, pm, o);
    }
    if (kGrad) {
      // Of entries with the same id, one writes the sum of their p: the one whose
      // number is left in the slice at that id.  (What the gradient's loop makes of
      // the numbers is written over.)
      __syncwarp();
      for (uint32_t k = lane; k < p.K; k += 32)
        if (e.id[k] >= 0) reinterpret_cast<Tag<E> *>(slice)[e.id[k] - e0] = (Tag<E>)k;
    }
    cluster_wait();  // every block of the cluster has started
    if (lane < (int)C)
      remote_store(remote_smem(&stats[rank], lane), make_float4(acc.m, acc.s, part, pm));
  } else {
    cluster_wait();
  }
  cluster_arrive();
  cluster_wait();
  acc = {stats[0].x, stats[0].y};
  for (uint32_t r = 1; r < C; ++r) acc = join(acc, {stats[r].x, stats[r].y}, p.scale);
  const float mass = mass_of_row;
  if (rank == 0 && tid == 0) {
    const float log_s = logf(acc.s);
    float loss = 0.0f;
    for (uint32_t r = 0; r < C; ++r) {
      const float4 v = stats[r];
      if (v.w != 0.0f)
        loss += v.z + v.w * fmaf(base_of(acc.m) - base_of(v.x), p.inv_temp, log_s);
    }
    // a student without any logit above -inf gives the teacher's entries probability 0
    if (acc.s == 0.0f) loss = mass == 0.0f ? 0.0f : -kNegInf;
    p.loss[row] = loss * p.temp * p.temp;
  }
  if (!kGrad) return;

  const float w = (p.weight ? p.weight[row] : 1.0f) * p.temp;
  const float f = acc.s == 0.0f ? 0.0f : w * mass / acc.s;  // of the exponentials
  const Ch<2> base = splat<2>(-base_of(acc.m)), by = splat<2>(f);
  if (mass == 0.0f) {  // no entry: nothing to learn, whatever the logits are
    for (uint32_t i = tid; i < mine; i += nthr) store_chunk(i, make_uint4(0, 0, 0, 0));
    return;
  }
#pragma unroll 2
  for (uint32_t i = tid; i < mine; i += nthr) {
    Ch<2> x[kN / 2];
    widen_chunk<E>(slice[i], x);
#pragma unroll
    for (int k = 0; k < kN / 2; ++k) {
      const Ch<2> y = (x[k] + base) * scale;
      x[k] = by * Ch<2>{exp2_sfu(y.v[0]), exp2_sfu(y.v[1])};
    }
    store_chunk(i, narrow_chunk<E>(x));
  }
  __syncthreads();  // the gradient is written
  if (warp == 0) {
    const Tag<E> *tags = reinterpret_cast<const Tag<E> *>(slice);
    bool twice = false;
    for (uint32_t k = lane; k < p.K; k += 32)
      if (e.id[k] >= 0 && tags[e.id[k] - e0] != (Tag<E>)k) twice = true;
    twice = __any_sync(0xffffffffu, twice);
    for (uint32_t k = lane; k < p.K; k += 32) {
      if (e.id[k] < 0 || tags[e.id[k] - e0] != (Tag<E>)k) continue;
      float pk = e.p[k];
      if (twice) {  // in the entries' order
        pk = 0.0f;
        for (uint32_t i = 0; i < p.K; ++i)
          if (e.id[i] == e.id[k]) pk += e.p[i];
      }
      const float g = f * exp2_sfu((e.x[k] - base_of(acc.m)) * p.scale);
      dst[e.id[k]] = from_f32<E>(fmaf(-w, pk, g));
    }
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
