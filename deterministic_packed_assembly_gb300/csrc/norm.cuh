// What the layer norm's kernels share (norm.cu has the choice among them).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "ring.cuh"
#include "rows.cuh"
#include "train.h"

namespace nsk {

constexpr uint32_t kNormSMs = 152;
constexpr uint32_t kFull = 0xffffffffu;
// Columns up to which a warp, or a part of one, has a row, without the ring: through it forward
// 131072 x 512 bf16 take 91 us in place of 79, 384 columns 94 in place of 77, backward 87 and 92
// in place of 89 and 86.  (Few rows of 512 columns backward are the other way: 700 in 9 us, 7
// through the ring.)
constexpr uint32_t kNormNarrow = 512;
constexpr uint32_t kNormWarps = 15;     // of a row, at most: with the one that copies 512 threads
constexpr uint32_t kNormKept = 5 * 32 * kOct * kNormWarps;  // columns that they have registers for
constexpr int kWideThreads = 512;       // of a row of more columns

struct NormParams {
  const void *x, *dy, *weight, *bias;
  bool floats;  // weight and bias are, whatever the rows
  int64_t x_row, dy_row;
  const int32_t *doc;
  void *y;  // or dx
  float *mean, *rstd;
  float eps;
  uint32_t N, D;
  uint32_t lanes, warps;  // of a row: lanes of one warp, or warps
  uint32_t stages;        // of the ring
  uint32_t fed;           // rows that come to it: N, but where a test withholds some
  float *partial;         // [blocks][2][D]
  void *dweight, *dbias;
  uint32_t blocks;
};

// How a row lies on threads, by its columns alone: what a row gets does not depend on
// the kernel that takes it.  nb spans a warp.  Forward a row's exchange of sums costs each of
// its warps the same, so that few are better while blocks are enough (32768 x 2560 bf16: ten
// warps 90 us, five 71), but weights take registers; backward the sums of the weights'
// gradients do, so that a warp has as few spans as 15 warps allow: 32768 x 2560 bf16 one span 90
// us, two 96, three 99; 32768 x 3584 one 119, two 127; 16384 x 4096 two 74, three 85; 8192 x
// 8192 three 78, five 122.
struct NormShape {
  uint32_t lanes, nb, warps;
};
inline NormShape norm_shape(uint32_t D, bool back) {
  NormShape s;
  s.lanes = lanes_for(D);
  const uint64_t spans = spans_for(D, s.lanes);
  if (D <= kNormNarrow) {
    s.nb = (uint32_t)spans, s.warps = 1;
    return s;
  }
  if (back)
    s.nb = spans <= kNormWarps ? 1 : spans <= 2 * kNormWarps ? 2 : spans <= 3 * kNormWarps ? 3 : 5;
  else
    s.nb = spans <= 5 ? 1 : spans <= 20 ? 2 : 5;
  s.warps = (uint32_t)((spans + s.nb - 1) / s.nb);
  return s;
}

// Columns that a row's threads have.
__host__ __device__ constexpr uint32_t norm_columns(uint32_t nb, uint32_t warps) {
  return nb * warps * 32 * kOct;
}

// Bytes of a block's weights in shared memory: those of more than three spans a warp, backward
// (besides their sums three spans' are what the registers hold).
__host__ __device__ constexpr uint32_t norm_kept(uint32_t nb, uint32_t warps, bool back) {
  return back && nb > 3 ? norm_columns(nb, warps) * (uint32_t)sizeof(float) : 0;
}

// The ring of rows of E on `warps` warps, NB spans each: as many of kBlocks blocks an SM as may be,
// batches of kMost to kLeast rows, as large as leave two stages; or no stages where two rows
// do not fit.
struct NormRing {
  uint32_t stages, rows, blocks;  // blocks an SM
  size_t shared;
};
template <class E, int NB, bool kBack, uint32_t kBlocks, uint32_t kMost, uint32_t kLeast>
constexpr NormRing norm_ring(uint32_t warps) {
  constexpr uint32_t kShared = 224 * 1024, kHead = 2 * 1024;  // of an SM; of a block besides
  const uint32_t slot = ring_slot(norm_columns(NB, warps), sizeof(E)) * (kBack ? 2 : 1);
  const uint32_t besides = norm_kept(NB, warps, kBack);
  for (uint32_t blocks = kBlocks; blocks > 0; --blocks)
    for (uint32_t rows = kMost; rows >= kLeast; rows /= 2) {
      const uint32_t room = kShared / blocks - 1024 - kHead - besides;
      const uint32_t stages = std::min(kRingStages, room / (slot * rows));
      if (stages >= 2) return {stages, rows, blocks, kHead + besides + (size_t)stages * rows * slot};
    }
  return {0, 0, 0, 0};
}
// Whether any of kFew to kWarps warps get batches of R rows: the kernels that are compiled.
template <class E, int NB, bool kBack, uint32_t kFew, uint32_t kWarps, uint32_t kBlocks,
          uint32_t kMost, uint32_t kLeast>
constexpr bool norm_ring_has(uint32_t R) {
  for (uint32_t warps = kFew; warps <= kWarps; ++warps)
    if (norm_ring<E, NB, kBack, kBlocks, kMost, kLeast>(warps).rows == R) return true;
  return false;
}

// Rows that a lane takes at once where a warp, or a part of one, has whole rows: 16
// registers of each array's.
template <class E, int NB, int V>
constexpr int kNormAtOnce =
    NB * Oct<E, V>::kPieces * Oct<E, V>::kWords > 8 ? 1 : 16 / (NB * Oct<E, V>::kPieces * Oct<E, V>::kWords);

// ---- sums over a row's lanes ------------------------------------------------------------
__device__ __forceinline__ float lanes_sum(float v, uint32_t lanes) {
  for (uint32_t o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
// Barrier of a group of warps.
__device__ __forceinline__ void group_sync(uint32_t group, uint32_t warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}
// K sums over `warps` warps (at most kWarps) at once, the same in every thread: lanes halve the values
// they add up as they halve their distance, in the order of lanes_sum.  part: [warps][K].
template <int K, int kWarps>
__device__ __forceinline__ void batch_sums(float (&v)[K], float *part, uint32_t warps,
                                           uint32_t warp, uint32_t lane) {
#pragma unroll
  for (int o = 16, n = K; o > 0; o >>= 1) {
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = lane & o ? v[i] : v[i + n], keep = lane & o ? v[i + n] : v[i];
        v[i] = keep + __shfl_xor_sync(kFull, give, o);
      }
    } else {
      v[0] += __shfl_xor_sync(kFull, v[0], o);
    }
  }
  // the value that is left is number (lane / (32 / K)) of them
  if (lane % (32 / K) == 0) part[warp * K + lane / (32 / K)] = v[0];
  group_sync(0, warps);
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < (int)warps) sum += part[w * K + lane % K];
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = __shfl_sync(kFull, sum, i);
}

// Eight columns of a weight vector, `otherwise` where there is none.
template <class E, int V>
__device__ __forceinline__ void load_vector(const void *p, bool floats, uint32_t c, uint32_t step,
                                            uint32_t D, float otherwise, Ch<2> (&v)[kOct / 2]) {
  if (p && floats) {
    Oct<float, V> x;
    clear(x);
    load_oct(x, static_cast<const float *>(p), c, step, D);
    widen(x, v);
  } else if (p) {
    Oct<E, V> x;
    clear(x);
    load_oct(x, static_cast<const E *>(p), c, step, D);
    widen(x, v);
  } else {
#pragma unroll
    for (int j = 0; j < kOct / 2; ++j) v[j] = splat<2>(otherwise);
  }
}

// Whether column j of a lane's eight is in the row.
template <int V>
__device__ __forceinline__ bool inside(uint32_t c, uint32_t step, uint32_t D, int j) {
  return c + j / V * step + j % V < D;
}

// The sum of v over a block, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float *sums) {
  v = lanes_sum(v, 32);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kWideThreads / 32; ++w) v += sums[w];
  return v;
}

// ---- the ring's two sides -----------------------------------------------------------------
// A row's statistics, and whether it is one that counts, beside it in the ring.
struct alignas(16) NormHead {
  float mean, rstd;
  uint32_t there, unused;
};
// Shared memory: barriers, heads, partial sums, and the rows.
struct NormShared {
  uint64_t full[kRingStages], empty[kRingStages];
  NormHead head[kRingStages][4];
  float part[2][kNormWarps * 8];
};
static_assert(sizeof(NormShared) <= 2 * 1024, "what norm_ring leaves for it");
constexpr uint32_t kNormRows = 2 * 1024;  // where the rows begin

__device__ __forceinline__ char *ring_row(char *rows, uint32_t stage, uint32_t array,
                                          uint32_t arrays, uint32_t R, uint32_t r, uint32_t slot) {
  return rows + ((stage * arrays + array) * R + r) * slot;
}

// The warp that copies: lane r has row r of each batch.  Documents and statistics are read a
// batch ahead, so that their way does not hold up the copies.  If a wait runs out it copies no
// more, and the others' waits run out too; a warp that has lost a batch leaves no stage any more,
// so that none is filled again before its copies have arrived.  The block ends after its
// copies, also where nobody waited for them.
template <class E, int R, bool kBack>
__device__ __forceinline__ void produce_rows(const NormParams &p, char *shared, char *rows,
                                             uint32_t slot) {
  NormShared &sh = *reinterpret_cast<NormShared *>(shared);
  const uint32_t lane = threadIdx.x % 32;
  constexpr uint32_t kArrays = kBack ? 2 : 1;
  if (lane >= R) return;
  const uint64_t every = (uint64_t)gridDim.x * R;
  uint64_t n = (uint64_t)blockIdx.x * R + lane;
  const auto look = [&](uint64_t i) {
    NormHead h = {0.0f, 0.0f, 0, 0};
    h.there = i < p.N && !(p.doc && p.doc[i] < 0);
    if (kBack && i < p.N) h.mean = p.mean[i], h.rstd = p.rstd[i];
    return h;
  };
  NormHead head = look(n);
  uint32_t stage = 0, turn = 0;
  for (; n - lane < p.fed; n += every) {
    const NormHead next = look(n + every);
    if (turn && !barrier_wait(&sh.empty[stage], (turn - 1) & 1)) break;
    sh.head[stage][lane] = head;
    RingSpan x = {0, 0, 0}, dy = x;
    char *xs = ring_row(rows, stage, 0, kArrays, R, lane, slot);
    char *ds = ring_row(rows, stage, kArrays - 1, kArrays, R, lane, slot);
    if (head.there) {
      x = ring_span(xs, static_cast<const E *>(p.x) + (int64_t)n * p.x_row, p.D, n == 0,
                    n + 1 == p.N);
      if (kBack)
        dy = ring_span(ds, static_cast<const E *>(p.dy) + (int64_t)n * p.dy_row, p.D, n == 0,
                       n + 1 == p.N);
    }
    barrier_expect(&sh.full[stage], x.bytes() + dy.bytes());  // arrives
    x.copy(xs, &sh.full[stage]);
    dy.copy(ds, &sh.full[stage]);
    head = next;
    if (++stage == p.stages) stage = 0, ++turn;
  }
  for (uint32_t i = 0; i < (turn ? p.stages : stage); ++i)
    barrier_wait(&sh.full[i], (i < stage ? turn : turn - 1) & 1);
}

// What every output of a batch comes to where a wait for it ran out.
__device__ __forceinline__ float norm_lost() { return __int_as_float(0x7fffffff); }

// A batch whose wait ran out (about a second): nothing is known of its heads, so that its rows are
// made to count as rows that are there, and its sums norm_lost().  (`lost` as a condition
// wherever a head is read, without the store: 16384 x 4096 bf16 forward 51 us in place of 48.)
template <int R>
__device__ __forceinline__ void lose_batch(NormShared &sh, uint32_t stage, uint32_t lane) {
  if (lane < R) sh.head[stage][lane].there = 1;
  __syncwarp(__activemask());
}

// Barriers, by the first thread; `warps` leave a stage.
template <int R>
__device__ __forceinline__ void start_ring(char *shared, uint32_t stages, uint32_t warps) {
  NormShared &sh = *reinterpret_cast<NormShared *>(shared);
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < stages; ++i) {
      barrier_init_count(&sh.full[i], R);
      barrier_init_count(&sh.empty[i], warps);
    }
    barrier_fence_init();
  }
  __syncthreads();
}

// ---- launches -----------------------------------------------------------------------
template <class E>
cudaError_t norm_forward(NormParams &p, int piece, cudaStream_t st);
template <class E>
cudaError_t norm_backward(NormParams &p, int piece, cudaStream_t st);

// By the pieces that all arrays can be moved by: for floats four elements at most, 16 bytes,
// which shared memory has in one access.
template <class E, class F>
cudaError_t norm_by_piece(int piece, F &&call) {
  constexpr int kMost = sizeof(E) == 4 ? 4 : 8;
  if (piece >= kMost) return call(std::integral_constant<int, kMost>{});
  if (piece >= 2) return call(std::integral_constant<int, 2>{});
  return call(std::integral_constant<int, 1>{});
}

}  // namespace nsk
