// Rows of a matrix streamed through shared memory by the bulk copy engine.
//
// One warp of a block issues the copies, R rows (a batch) to a stage of the ring, and the others
// compute: a batch is taken when its bytes have arrived (`full`, counted by the copies),
// and its stage is filled again when every warp has left it (`empty`).  A row may begin
// anywhere: the whole 16-byte pieces that hold it are copied, so that it lies in shared memory
// as it lies in memory, off a boundary by the same few bytes.  Only at an array's
// two ends, where such a piece would reach beyond it, single elements are copied instead.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"
#include "rows.cuh"

namespace nsk {

constexpr uint32_t kRingStages = 8;  // at most

__device__ __forceinline__ void barrier_init_count(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(bar)),
               "r"(count)
               : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(bar))
               : "memory");
}
// Inits are visible to the copy engine.
__device__ __forceinline__ void barrier_fence_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// `bytes` (a multiple of 16) from global to shared memory, both on 16-byte boundaries; they are
// counted down at `bar`.
__device__ __forceinline__ void bulk_copy(void *smem, const void *gmem, uint32_t bytes,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"((uint32_t)__cvta_generic_to_shared(smem)),
      "l"(gmem), "r"(bytes), "r"((uint32_t)__cvta_generic_to_shared(bar))
      : "memory");
}

// Bytes of a row's place in the ring, for as many columns as its threads read.
__host__ __device__ constexpr uint32_t ring_slot(uint32_t columns, uint32_t es) {
  return (columns * es + 30) / 16 * 16;
}

// The part of a row that the engine copies, from `lo` to `hi`.
struct RingSpan {
  uintptr_t lo, hi, base;
  __device__ __forceinline__ uint32_t bytes() const { return (uint32_t)(hi - lo); }
  __device__ __forceinline__ void copy(char *slot, uint64_t *bar) const {
    if (hi > lo) bulk_copy(slot + (lo - base), reinterpret_cast<const void *>(lo), bytes(), bar);
  }
};
// Of a row of D elements; what is not in it is copied here and now.  `first` and `last`:
// nothing before, or behind, the row belongs to the array.
template <class E>
__device__ __forceinline__ RingSpan ring_span(char *slot, const E *row, uint32_t D, bool first,
                                              bool last) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(row), b = a + (uint64_t)D * sizeof(E);
  RingSpan s;
  s.base = a & ~(uintptr_t)15;
  s.lo = first ? (a + 15) & ~(uintptr_t)15 : s.base;
  s.hi = last ? b & ~(uintptr_t)15 : (b + 15) & ~(uintptr_t)15;
  if (s.hi < s.lo) s.lo = s.hi = b;
  for (uintptr_t i = a; i < s.lo; i += sizeof(E))
    *reinterpret_cast<E *>(slot + (i - s.base)) = *reinterpret_cast<const E *>(i);
  for (uintptr_t i = s.hi; i < b; i += sizeof(E))
    *reinterpret_cast<E *>(slot + (i - s.base)) = *reinterpret_cast<const E *>(i);
  // later copies of the engine to the same place come after these
  if (a < s.lo || s.hi < b) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  return s;
}

// A lane's eight columns of a row in the ring, pieces 32 V columns apart; what lies behind the
// row is read too, and comes to nothing by `only`.
template <class E, int V>
__device__ __forceinline__ void ring_oct(Oct<E, V> &x, const char *at) {
  using O = Oct<E, V>;
#pragma unroll
  for (int i = 0; i < O::kPieces; ++i) {
    uint32_t *w = x.w + i * O::kWords;
    const char *p = at + i * 32 * V * (int)sizeof(E);
    if constexpr (O::kBytes >= 16) {
#pragma unroll
      for (int j = 0; j < O::kWords / 4; ++j) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[j];
        w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
      }
    } else if constexpr (O::kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (O::kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
}
// Columns c, c + 32 V, ... of V each; those beyond D become 0.
template <class E, int V>
__device__ __forceinline__ void only(Oct<E, V> &x, uint32_t c, uint32_t D) {
  using O = Oct<E, V>;
#pragma unroll
  for (int i = 0; i < O::kPieces; ++i)
    if (c + i * 32 * V >= D) {
#pragma unroll
      for (int j = 0; j < O::kWords; ++j) x.w[i * O::kWords + j] = 0;
    }
}
// The eight columns to a row of which all lanes' are there.
template <class E, int V>
__device__ __forceinline__ void store_all(E *at, const Oct<E, V> &x) {
  using O = Oct<E, V>;
#pragma unroll
  for (int i = 0; i < O::kPieces; ++i)
    store_piece<O::kBytes>(at + i * 32 * V, x.w + i * O::kWords);
}

}  // namespace nsk
