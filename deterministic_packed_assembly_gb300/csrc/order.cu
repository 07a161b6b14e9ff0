// A stable sort of small whole numbers by counting: one pass a digit, the lowest first.
//
// A first kernel counts the lowest digits of each block's stretch of keys (R counters a
// block).  Then a kernel a pass: every block adds up the counters of all blocks itself (at
// most 152 x R words, from the L2 cache: a kernel between the two would cost its
// launch), so that it knows where its own keys of each digit go; a warp takes a
// contiguous part of the stretch, 32 keys at a time, and its lanes with the same digit
// rank themselves by a match.  As it places a key it counts the key's next digit for the
// stretch that the key will lie in.  Counts are whole numbers: atomics do not change them,
// and equal keys keep their order.
//
// What bounds it is latency: a launch and some trips to the L2 cache a pass.  The first pass
// reads its keys while the counters are still being made.  32768 tokens of 128256: 17 us;
// 262144 choices of 64 experts 9, 1048576 of 256 21.  (One block for few keys, all passes in
// shared memory, was slower from 1000 keys on: 8192 in 38 us in place of 15.)

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "order.h"
#include "train.h"

namespace nsk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kMostBlocks = 152;
constexpr uint32_t kNone = 0xffffffffu;
constexpr int kAhead = 8;  // keys a thread has under way

struct Pass {
  Keys keys;
  const Sorted *from;  // the pass before's, or null: the keys themselves
  Sorted *to;          // or null: place and slots
  int32_t *place, *slots, *offsets;
  uint8_t *used;       // first pass
  uint32_t *counter;
  uint32_t *table;     // [blocks][rounded_digits(R)]
  uint32_t *after;     // the next pass's, or null
  uint32_t passes;     // tables, of which the first kernel clears all but the first
  uint32_t R, shift, mask, stretch, bits;
};

__host__ __device__ __forceinline__ uint32_t rounded_digits(uint32_t R) { return (R + 3) / 4 * 4; }

// Tables of one pass.
__host__ __device__ __forceinline__ uint64_t table_words(uint32_t blocks, uint32_t R) {
  return (uint64_t)blocks * rounded_digits(R);
}

// From the L2 cache: what the kernel before wrote may be read while the one between them runs.
__device__ __forceinline__ Sorted key_at(const Pass &p, uint32_t i) {
  if (p.from) {
    const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(p.from) + i);
    return {v.x, v.y};
  }
  const int64_t id = p.keys.wide ? static_cast<const int64_t *>(p.keys.ids)[i]
                                 : static_cast<const int32_t *>(p.keys.ids)[i];
  const bool there =
      id >= 0 && id < (int64_t)p.keys.limit && !(p.keys.doc && p.keys.doc[i] < 0);
  return {there ? (uint32_t)id : p.keys.limit, i};
}

__global__ void __launch_bounds__(kThreads) count_kernel(const Pass p) {
  extern __shared__ uint32_t count[];
  for (uint32_t d = threadIdx.x; d < p.R; d += kThreads) count[d] = 0;
  pdl_wait_then_release();
  const uint32_t Rp = rounded_digits(p.R), all = gridDim.x * kThreads;
  const uint32_t self = blockIdx.x * kThreads + threadIdx.x;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (p.used) {
    for (uint32_t i = self; i < p.keys.limit / 16 + 1; i += all)
      reinterpret_cast<uint4 *>(p.used)[i] = zero;
    if (self == 0) *p.counter = 0;
  }
  const uint64_t quads = table_words(gridDim.x, p.R) / 4;
  for (uint64_t i = quads + self; i < quads * p.passes; i += all)
    reinterpret_cast<uint4 *>(p.table)[i] = zero;
  __syncthreads();
  const uint32_t begin = blockIdx.x * p.stretch;
  const uint32_t end = min(p.keys.N, begin + p.stretch);
  for (uint32_t i0 = begin + threadIdx.x; i0 < end; i0 += kThreads * kAhead) {
    uint32_t key[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i0 + a * kThreads < end) key[a] = key_at(p, i0 + a * kThreads).key;
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i0 + a * kThreads < end) atomicAdd(&count[(key[a] >> p.shift) & p.mask], 1u);
  }
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < Rp; d += kThreads)
    p.table[(uint64_t)blockIdx.x * Rp + d] = d < p.R ? count[d] : 0;
}

__global__ void __launch_bounds__(kThreads) place_kernel(const Pass p) {
  extern __shared__ uint32_t shared[];
  const uint32_t Rp = rounded_digits(p.R);
  uint32_t *total = shared;              // [R]: of all blocks, then the digits before
  uint32_t *before = total + Rp;         // [R]: of the blocks before this one
  uint32_t *start = before + Rp;         // [kWarps][R]
  __shared__ uint32_t sums[kWarps];
  const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (uint32_t d = threadIdx.x; d < 2 * Rp + kWarps * p.R; d += kThreads) shared[d] = 0;
  __syncthreads();
  if (p.from) pdl_wait();

  // this warp's own digits; few keys stay in registers
  const uint32_t part = p.stretch / kWarps;
  const uint32_t begin = min(p.keys.N, blockIdx.x * p.stretch + warp * part);
  const uint32_t end = min(p.keys.N, begin + part);
  uint32_t *mine = start + warp * p.R;
  Sorted key[kAhead];
  const auto load = [&](uint32_t i0) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i0 + 32 * a + lane < end) key[a] = key_at(p, i0 + 32 * a + lane);
  };
  for (uint32_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
    load(i0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (i0 + 32 * a + lane < end) atomicAdd(&mine[(key[a].key >> p.shift) & p.mask], 1u);
  }
  if (!p.from) pdl_wait();
  release_dependents();
  // all blocks' counters: neighbouring threads take four neighbouring digits each, groups of
  // them share the blocks
  const uint32_t quads = Rp / 4, groups = kThreads / min(quads, (uint32_t)kThreads);
  const uint32_t group = threadIdx.x / quads;
  if (group < groups) {
    const uint4 *table = reinterpret_cast<const uint4 *>(p.table);
    const uint32_t d = threadIdx.x % quads;
    uint4 all = make_uint4(0, 0, 0, 0), ahead = all;
#pragma unroll 8
    for (uint32_t b = group; b < gridDim.x; b += groups) {
      const uint4 c = __ldcg(table + (uint64_t)b * quads + d);
      all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
      if (b < blockIdx.x) ahead.x += c.x, ahead.y += c.y, ahead.z += c.z, ahead.w += c.w;
    }
    atomicAdd(&total[4 * d], all.x), atomicAdd(&before[4 * d], ahead.x);
    atomicAdd(&total[4 * d + 1], all.y), atomicAdd(&before[4 * d + 1], ahead.y);
    atomicAdd(&total[4 * d + 2], all.z), atomicAdd(&before[4 * d + 2], ahead.z);
    atomicAdd(&total[4 * d + 3], all.w), atomicAdd(&before[4 * d + 3], ahead.w);
  }
  __syncthreads();
  // digits before: each thread has a run of them
  const uint32_t run = (p.R + kThreads - 1) / kThreads;
  const uint32_t d0 = min(p.R, threadIdx.x * run), d1 = min(p.R, d0 + run);
  uint32_t sum = 0;
  for (uint32_t d = d0; d < d1; ++d) sum += total[d];
  uint32_t scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= (uint32_t)o) scan += v;
  }
  if (lane == 31) sums[warp] = scan;
  __syncthreads();
  uint32_t base = scan - sum;
#pragma unroll
  for (uint32_t w = 0; w < kWarps; ++w) base += w < warp ? sums[w] : 0;
  for (uint32_t d = d0; d < d1; ++d) {
    if (p.offsets && blockIdx.x == 0) p.offsets[d] = (int32_t)base;
    uint32_t c[kWarps], at = base + before[d];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) c[w] = start[w * p.R + d];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      start[w * p.R + d] = at;
      at += c[w];
    }
    base += total[d];
  }
  __syncthreads();

  for (uint32_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
    if (part > 32 * kAhead) load(i0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (i0 + 32 * a >= end) break;
      const uint32_t i = i0 + 32 * a + lane, k = key[a].key;
      const uint32_t d = i < end ? (k >> p.shift) & p.mask : kNone;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      const uint32_t rank = __popc(same & ((1u << lane) - 1));
      // a token that many positions have is marked once a warp
      const uint32_t leader = __shfl_sync(0xffffffffu, k, __ffs(same) - 1);
      uint32_t at = 0;
      if (i < end) at = mine[d] + rank;
      __syncwarp();
      if (i < end && rank == 0) mine[d] += __popc(same);
      __syncwarp();
      if (i >= end) continue;
      if (p.used && k < p.keys.limit && (rank == 0 || k != leader)) p.used[k] = 1;
      if (p.to) {
        p.to[at] = key[a];
        if (p.after)
          atomicAdd(p.after + (uint64_t)(at / p.stretch) * Rp + ((k >> (p.shift + p.bits)) & p.mask),
                    1u);
      } else {
        p.place[i] = (int32_t)at;
        p.slots[at] = (int32_t)i;
      }
    }
  }
}

// Keys of a block's stretch: as few blocks as fill the SMs, a multiple of 32 a warp.
uint32_t stretch_of(uint32_t N) {
  const uint32_t each = (N + kMostBlocks - 1) / kMostBlocks;
  return std::max<uint32_t>(1, (each + kThreads - 1) / kThreads) * kThreads;
}
uint32_t blocks_of(uint32_t N) {
  const uint32_t s = stretch_of(N);
  return std::max<uint32_t>(1, (N + s - 1) / s);
}

cudaError_t launch_count(const Pass &p, cudaStream_t st) {
  const cudaError_t e = allow_shared_memory(reinterpret_cast<const void *>(place_kernel));
  if (e != cudaSuccess) return e;
  ++launch_counter();
  count_kernel<<<blocks_of(p.keys.N), kThreads, p.R * sizeof(uint32_t), st>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_place(const Pass &p, cudaStream_t st) {
  const size_t shared = (2 * rounded_digits(p.R) + kWarps * (size_t)p.R) * sizeof(uint32_t);
  ++launch_counter();
  pdl_launch(place_kernel, dim3(blocks_of(p.keys.N)), dim3(kThreads), shared, st, p);
  return cudaGetLastError();
}

// Digits of the keys 0 to limit: passes of at most nine bits.
struct Digits {
  uint32_t passes, bits;
};
Digits digits_of(uint32_t limit) {
  uint32_t bits = 1;
  while (bits < 32 && (limit >> bits)) ++bits;
  const uint32_t passes = (bits + 8) / 9;
  return {passes, (bits + passes - 1) / passes};
}
uint64_t rounded(uint64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

uint64_t order_choices_workspace(uint32_t N, uint32_t limit) {
  return table_words(blocks_of(N), limit + 1) * sizeof(uint32_t);
}

cudaError_t launch_order_choices(const Keys &keys, int32_t *place, int32_t *slots,
                                 int32_t *offsets, void *workspace, cudaStream_t st) {
  Pass p = {};
  p.keys = keys, p.place = place, p.slots = slots, p.offsets = offsets;
  p.table = static_cast<uint32_t *>(workspace), p.passes = 1;
  p.R = keys.limit + 1, p.shift = 0, p.mask = kNone, p.stretch = stretch_of(keys.N);
  const cudaError_t e = launch_count(p, st);
  return e == cudaSuccess ? launch_place(p, st) : e;
}

uint64_t order_tokens_workspace(uint32_t N, uint32_t limit) {
  const Digits d = digits_of(limit);
  return rounded(d.passes * table_words(blocks_of(N), 1u << d.bits) * sizeof(uint32_t)) +
         (d.passes > 1 ? (uint64_t)N * sizeof(Sorted) : 0);
}

cudaError_t launch_order_tokens(const Keys &keys, Sorted *sorted, uint8_t *used,
                                uint32_t *counter, void *workspace, cudaStream_t st) {
  const Digits d = digits_of(keys.limit);
  const uint64_t words = table_words(blocks_of(keys.N), 1u << d.bits);
  Sorted *other = reinterpret_cast<Sorted *>(static_cast<char *>(workspace) +
                                             rounded(d.passes * words * sizeof(uint32_t)));
  Pass p = {};
  p.keys = keys, p.table = static_cast<uint32_t *>(workspace), p.passes = d.passes;
  p.R = 1u << d.bits, p.mask = p.R - 1, p.bits = d.bits, p.stretch = stretch_of(keys.N);
  p.used = used, p.counter = counter;
  cudaError_t e = launch_count(p, st);
  for (uint32_t i = 0; i < d.passes && e == cudaSuccess; ++i) {
    p.shift = i * d.bits;
    p.from = i == 0 ? nullptr : p.to;
    p.to = (d.passes - i) % 2 ? sorted : other;  // the last pass writes `sorted`
    p.used = i == 0 ? used : nullptr;
    if (i) p.table += words;
    p.after = i + 1 < d.passes ? p.table + words : nullptr;
    e = launch_place(p, st);
  }
  return e;
}

}  // namespace nsk
