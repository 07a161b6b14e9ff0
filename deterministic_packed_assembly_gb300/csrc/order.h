// A stable sort of small whole numbers (internal interface of order.cu): tokens by
// their id for the gradient of a table, choices of experts by expert.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace nsk {

// Keys are ids in [0, limit); an id outside, or whose doc is below 0, has the key `limit`
// and so comes last.
struct Keys {
  const void *ids;     // int32, or int64 where `wide`
  const int32_t *doc;  // or null
  uint32_t N;          // below 2^31
  uint32_t limit;      // below 2^31
  bool wide;
};

// A position in the order: a key and where it was.
struct alignas(8) Sorted {
  uint32_t key, at;
};

// Choices by expert, in one pass (keys.limit <= 1024): place[i] is choice i's place, slots its
// inverse, offsets[e] how many choices come before expert e's.
uint64_t order_choices_workspace(uint32_t N, uint32_t limit);
cudaError_t launch_order_choices(const Keys &keys, int32_t *place, int32_t *slots,
                                 int32_t *offsets, void *workspace, cudaStream_t st);

// Tokens by id: `sorted` receives N positions, used[id] (rounded up to 16 bytes) 1 where the
// id is there and else 0, and *counter 0.
uint64_t order_tokens_workspace(uint32_t N, uint32_t limit);
cudaError_t launch_order_tokens(const Keys &keys, Sorted *sorted, uint8_t *used,
                                uint32_t *counter, void *workspace, cudaStream_t st);

}  // namespace nsk
