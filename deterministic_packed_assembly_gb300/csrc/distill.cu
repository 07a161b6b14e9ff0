// Distillation from a teacher's top logits: the loss of every row and the
// gradient of its logits, in one pass over them.
//
//   q = softmax(s / temp) over V, p from the teacher's K entries, m = sum p
//   loss = temp^2 sum_k p_k (log p_k - log q_k),  ds_v = w temp (m q_v - p_v)
//
// The gradient needs the row's softmax sum before its first element can be
// written, and a row (256 KB for a vocabulary of 128K in 16 bits) is read from
// memory once: a cluster of C blocks keeps the row in its shared memory, a slice
// each.  A thread has its own 16-byte chunks of the slice: it copies them in
// asynchronously, reduces them to a reference and a sum as they arrive, and,
// once the blocks have exchanged theirs, turns each into the gradient and starts
// the copy of the cluster's next row into its place.  So the copies of a row run
// beside the stores of the one before.  The teacher's K entries are few: two
// warps of their own in each block have them, of even and of odd rows, ahead of the
// rows' warps: what they do for a row is a chain of loads that takes as long as one or
// two rows, so that each loads its next row's entries while statistics are exchanged.
// With c the student's logit at the teacher's first choice, M and S the row's maximum
// and sum,
//   temp sum_k p_k (log p_k - log q_k) = sum_k p_k (temp log p_k - (s_k - c))
//                                        + m (temp log S + (M - c)),
// (not divided by temp: a choice whose logit is near the type's lowest value has a large
// loss, not an infinity less another).  The first sum each block takes over the ids in
// its slice, without the row's statistics, so that one exchange is enough; its terms are
// small, as the teacher's choices are near c.  After the gradient is written their warp
// writes the entries' own over it.
//
// Logits are kept as they came.  An exponential is 2^((s - max) log2 e / temp):
// the difference is taken first, so that it is exact where it matters, near the
// maximum, and a row at the type's lowest value does not overflow.
//
// Bound by memory where the gradient is wanted (8192 x 128256 bfloat16, 65 % of the rows
// learned: 565 us, 6.15 TB/s, 0.90 of a copy's bandwidth), by the SMs' instructions where
// it is not (4093 x 50257: 76 us, 63 % of the issue slots, 5.1 TB/s), by the entries'
// chain where K is large (1021 x 50257 float: 93 us with K = 200, 75 us with 16).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "train.h"

namespace nsk {
namespace {

constexpr int kEntryWarps = 2;  // one for even rows, one for odd ones
constexpr int kMaxThreads = 256 + 32 * kEntryWarps;
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
  bool same;                    // every row starts at the same place of 16 bytes
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

// A reference (-inf at first), and the sum of exp((x - reference) / temp).  The
// reference is one of the logits and no more than a few powers of two below the
// largest so far: it is raised only when a chunk's sum passes kFarAbove, so that the
// maximum of every chunk need not be found; an exponent's rounding stays that of a
// number of a few units.
constexpr float kFarAbove = 256.0f;
struct MaxSum {
  float m, s;
};
// What is taken from x: the reference, where -inf leaves x = -inf alone.
__device__ __forceinline__ float base_of(float m) { return m == kNegInf ? 0.0f : m; }
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float scale) {
  MaxSum r;
  r.m = fmaxf(a.m, b.m);
  const float base = base_of(r.m);
  r.s = a.s * exp2_sfu((a.m - base) * scale) + b.s * exp2_sfu((b.m - base) * scale);
  return r;
}

template <class E>
__device__ __forceinline__ float chunk_max(uint4 v) {
  Ch<2> x[8 / sizeof(E)];
  widen_chunk<E>(v, x);
  float top = fmaxf(x[0].v[0], x[0].v[1]);
#pragma unroll
  for (int k = 1; k < (int)(8 / sizeof(E)); ++k) top = fmaxf(top, fmaxf(x[k].v[0], x[k].v[1]));
  return top;
}
// Sum of 2^((x + minus) scale).
template <class E>
__device__ __forceinline__ float chunk_sum(uint4 v, float minus, Ch<2> scale) {
  Ch<2> x[8 / sizeof(E)], sum;
  widen_chunk<E>(v, x);
#pragma unroll
  for (int k = 0; k < (int)(8 / sizeof(E)); ++k) {
    const Ch<2> y = (x[k] + splat<2>(minus)) * scale;
    const Ch<2> e = {exp2_sfu(y.v[0]), exp2_sfu(y.v[1])};
    sum = k == 0 ? e : sum + e;
  }
  return sum.v[0] + sum.v[1];
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

// A row of logits: `head` elements, then whole chunks of 16 bytes from a 16-byte
// boundary on, then the rest, which is shorter than a chunk.  This block's slice is
// `mine` of the chunks; the first one starts at element `from`.  The elements at
// both ends are the first block's entry warp's, one or none a lane.
template <class E>
struct RowSlice {
  static constexpr int kN = 16 / sizeof(E);  // elements of a chunk
  int head, tail;  // the tail's first element
  int from;
  uint32_t mine;
  __device__ __forceinline__ RowSlice(const DistillParams &p, uint32_t row, uint32_t rank) {
    const uintptr_t at = (uintptr_t)(static_cast<const E *>(p.logits) + (int64_t)row * p.logits_row);
    head = min((int)(((16 - (at & 15)) & 15) / sizeof(E)), (int)p.V);
    const uint32_t chunks = (p.V - head) / kN;
    const uint32_t first = min(rank * p.slice, chunks);
    mine = min(p.slice, chunks - first);
    from = head + (int)(first * kN);
    tail = head + (int)(chunks * kN);
  }
  // The element at the row's ends that a lane of the entry warp has, -1 for none.
  __device__ __forceinline__ int end_of(const DistillParams &p, uint32_t rank, int lane) const {
    const int i = lane < kN ? lane : tail + lane - kN;
    return rank == 0 && (lane < kN ? i < head : lane < 2 * kN && i < (int)p.V) ? i : -1;
  }
};

// A row's ids and teacher logits into the L2 cache: read from memory beside the rows'
// copies they take microseconds.
__device__ __forceinline__ void prefetch_entries(const DistillParams &p, uint32_t row, int lane) {
  const uint64_t ids = (uint64_t)p.K * (p.ids_64 ? 8 : 4),
                 top = (uint64_t)p.K * (p.top_dtype == NS_F32 ? 4 : 2);
  const char *a = static_cast<const char *>(p.ids) + row * ids,
             *b = static_cast<const char *>(p.top) + row * top;
  for (uint64_t i = (uint64_t)lane * 128; i < ids; i += 32 * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a + i));
  for (uint64_t i = (uint64_t)lane * 128; i < top; i += 32 * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(b + i));
}

// A row's ids and teacher logits into `e`, by lanes; its largest teacher logit, the
// first of them and its id.
struct Teacher {
  float m, lse;
  uint32_t top;  // 0xffffffff: no entry
  int top_id;
};
__device__ __forceinline__ Teacher load_teacher(const DistillParams &p, uint32_t row, int lane,
                                                int *ids, float *logits) {
  const int64_t base = (int64_t)row * p.K;
  Teacher r = {kNegInf, p.teacher_lse ? p.teacher_lse[row] : 0.0f, 0xffffffffu, 0};
#pragma unroll 4
  for (uint32_t k = lane; k < p.K; k += 32) {
    const int64_t v = p.ids_64 ? static_cast<const int64_t *>(p.ids)[base + k]
                               : (int64_t)static_cast<const int32_t *>(p.ids)[base + k];
    const float t = load_top(p.top, p.top_dtype, base + k);
    const int id = v >= 0 && v < (int64_t)p.V ? (int)v : -1;
    ids[k] = id;
    logits[k] = id >= 0 ? t : kNegInf;
    if (id >= 0 && t > r.m) r.m = t, r.top = k, r.top_id = id;
  }
  return r;
}

// The entries' warp: the teacher's probabilities and the student's logits at the
// entries of this block's slice [from, to).
struct EntrySums {
  float mass;  // sum of p over the row: 1 unless the teacher's own normaliser is given
  float c;     // the student's logit at the teacher's first choice
  float part;  // sum of p (temp log p - (s - c)) over the slice
};
template <class E>
__device__ __forceinline__ EntrySums teacher_entries(const DistillParams &p,
                                                     const E *logits, const RowSlice<E> &s,
                                                     uint32_t rank, int lane, const Entries &e,
                                                     const Teacher &teacher) {
  // an id is this block's: in its chunks, or at the row's ends for the first block
  const int last = s.from + (int)s.mine * (16 / (int)sizeof(E));
  auto ours = [&](int id) {
    return (id >= s.from && id < last) || (rank == 0 && id >= 0 && (id < s.head || id >= s.tail));
  };
  float m = teacher.m;
  uint32_t top = teacher.top;
  int top_id = teacher.top_id;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o);
    const uint32_t ok = __shfl_xor_sync(0xffffffffu, top, o);
    const int oi = __shfl_xor_sync(0xffffffffu, top_id, o);
    if (om > m || (om == m && ok < top)) m = om, top = ok, top_id = oi;
  }
  EntrySums r = {0.0f, 0.0f, 0.0f};
  E at_top = from_f32<E>(0.0f);
  if (top != 0xffffffffu) at_top = logits[top_id];
  constexpr int kBatch = 8;  // loads in flight
  for (uint32_t k0 = lane; k0 < p.K; k0 += 32 * kBatch) {
    E x[kBatch];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t k = k0 + 32 * i;
      const int id = k < p.K ? e.id[k] : -1;
      if (ours(id)) x[i] = logits[id], mine |= 1u << i;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (mine >> i & 1) e.x[k0 + 32 * i] = to_f32(x[i]);
  }
  // The exchange waits for the value itself: its logit may be in another block's slice,
  // which writes the gradient there, perhaps over the logits, as soon as this block has
  // sent its sums, and no store waits for a load whose value nothing has used.
  r.c = __shfl_sync(0xffffffffu, to_f32(at_top), 0);
  if (r.c == kNegInf) r.c = 0.0f;
  const float base_m = base_of(m);
  float sum = 0.0f;
#pragma unroll 2
  for (uint32_t k = lane; k < p.K; k += 32) {
    const float t = e.logp[k];
    const float l = p.teacher_lse ? fmaf(t, p.inv_temp, -teacher.lse) : (t - base_m) * p.inv_temp;
    // an absent entry stays at -inf whatever lse is
    const float keep = e.id[k] < 0 ? kNegInf : l;
    const float v = expf(keep);
    e.logp[k] = keep;
    e.p[k] = v;
    sum += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float inv = 1.0f, log_sum = 0.0f;
  r.mass = sum;
  if (!p.teacher_lse && sum != 0.0f)
    inv = 1.0f / sum, log_sum = logf(sum), r.mass = sum == sum ? 1.0f : sum;  // or a NaN
#pragma unroll 2
  for (uint32_t k = lane; k < p.K; k += 32) {
    const int id = e.id[k];
    if (!ours(id)) {
      e.id[k] = -1;  // absent, or another block's
      continue;
    }
    const float pk = e.p[k] * inv, x = e.x[k];
    e.p[k] = pk;
    if (pk != 0.0f)
      r.part += pk * (x == kNegInf ? -kNegInf : fmaf(p.temp, e.logp[k] - log_sum, r.c - x));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.part += __shfl_xor_sync(0xffffffffu, r.part, o);
  return r;
}

// Of a slice's entries with the same id the first one is to write the gradient, of
// the sum of their p (in the entries' order); the others' ids become -1.  `seen` has
// kSeen bits, 0 before and after, that an id's hash picks from: an id that finds its
// bit set is looked for among the others.
constexpr uint32_t kSeen = 4096;
__device__ __forceinline__ uint32_t bit_of(int id) {  // Knuth's multiplicative hash
  return (uint32_t)id * 2654435761u >> 20;
}
static_assert(kSeen == 1u << (32 - 20), "a hash is a bit's number");
static_assert(NS_DISTILL_MAX_TOP <= 32 * 32, "a lane's entries are a word's bits");
__device__ void join_repeated(uint32_t K, int lane, const Entries &e, uint32_t *seen) {
  uint32_t again = 0;  // this lane's entries (k / 32) that found their bit set
  for (uint32_t k = lane, i = 0; k < K; k += 32, ++i) {
    const int id = e.id[k];
    if (id < 0) continue;
    const uint32_t h = bit_of(id), bit = 1u << (h & 31);
    if (atomicOr(&seen[h >> 5], bit) & bit) again |= 1u << i;
  }
  __syncwarp();
  for (uint32_t k = lane; k < K; k += 32)
    if (e.id[k] >= 0) seen[bit_of(e.id[k]) >> 5] = 0;
  bool twice = false;
  for (uint32_t lanes; (lanes = __ballot_sync(0xffffffffu, again != 0)) != 0;) {
    const int from = __ffs(lanes) - 1;  // the warp looks for one of this lane's
    const int id = __shfl_sync(0xffffffffu, again ? e.id[lane + 32 * (__ffs(again) - 1)] : 0, from);
    if (lane == from) again &= again - 1;
    int found = 0;
    for (uint32_t k = lane; k < K; k += 32) found += e.id[k] == id;
    if (__reduce_add_sync(0xffffffffu, found) > 1) twice = true;
  }
  __syncwarp();
  if (!twice) return;
  for (uint32_t k = lane; k < K; k += 32) {
    const int id = e.id[k];
    if (id < 0) continue;
    float sum = -1.0f;  // no sum of probabilities: not the first
    uint32_t i = 0;
    while (e.id[i] != id) ++i;
    if (i == k) {
      sum = 0.0f;
      for (; i < K; ++i)
        if (e.id[i] == id) sum += e.p[i];
    }
    e.logp[k] = sum;  // the loss is done with the logarithms
  }
  __syncwarp();
  for (uint32_t k = lane; k < K; k += 32) {
    if (e.id[k] < 0) continue;
    if (e.logp[k] == -1.0f) e.id[k] = -1;
    else e.p[k] = e.logp[k];
  }
}

// Gradients whose chunks do not lie on 16-byte boundaries.
template <class E>
__device__ __noinline__ void store_apart(E *to, uint4 v) {
  E x[16 / sizeof(E)];
  *reinterpret_cast<uint4 *>(x) = v;
#pragma unroll
  for (int k = 0; k < (int)(16 / sizeof(E)); ++k) to[k] = x[k];
}
template <class E>
__device__ __forceinline__ void store_chunk(E *to, bool wide, uint4 v) {
  if (wide) *reinterpret_cast<uint4 *>(to) = v;
  else store_apart<E>(to, v);
}

// The cluster's rows: its number, and every `stride`-th one from there.  `mask` is
// read for 32 of them at once, a lane each.
struct RowWalk {
  uint32_t next, stride, bits, left;  // bits of the `left` rows from `next` on
  __device__ __forceinline__ RowWalk(uint32_t first, uint32_t s) : next(first), stride(s) {
    bits = left = 0;
  }
  // The next learned row (N: there is none); `skipped` is called with each row before.
  template <class F>
  __device__ __forceinline__ uint32_t learned(const DistillParams &p, int lane, F skipped) {
    while (next < p.N) {
      if (left == 0) {
        const uint64_t r = next + (uint64_t)lane * stride;
        bits = __ballot_sync(0xffffffffu, r < p.N && (!p.mask || p.mask[r] != 0));
        left = 32;
      }
      const uint32_t row = next;
      const bool is = bits & 1u;
      bits >>= 1, --left;
      next = stride < p.N - next ? next + stride : p.N;
      if (is) return row;
      skipped(row);
    }
    return p.N;
  }
};

// Statistics of rows on their way between the blocks: a row's place is written again
// four rows later.  By then every reader has read it: a block's statistics of row i
// + 4 are sent when those of row i + 3, and so of row i + 2, are complete, which
// every entry warp sends after it has read those of row i.
constexpr int kPlaces = 4;
struct Shared {
  float4 stats[kPlaces][kMaxCluster];  // every slice's maximum, sum and part, the row's mass
  uint64_t arrived[kPlaces];           // mbarriers: the stats have
  float2 warp_stats[2][kMaxThreads / 32];
};

// Barriers 1 and 2: an even or odd row's gradient is written; 3 and 4: its
// warp_stats are.  The rows' warps only arrive, one entry warp waits.
__device__ __forceinline__ int row_threads() { return blockDim.x - 32 * kEntryWarps; }
__device__ __forceinline__ void named_arrive(int barrier) {
  asm volatile("bar.arrive %0, %1;" ::"r"(barrier), "r"(row_threads() + 32) : "memory");
}
__device__ __forceinline__ void named_wait(int barrier) {
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(row_threads() + 32) : "memory");
}
__device__ __forceinline__ bool stats_wait(Shared &sh, uint32_t round) {
  return barrier_wait(&sh.arrived[round % kPlaces], round / kPlaces & 1);
}

struct RowStats {
  MaxSum all;
  float parts, mass;
};
__device__ __forceinline__ RowStats row_stats(const DistillParams &p, Shared &sh, uint32_t round,
                                              uint32_t C, bool &lost) {
  if (!lost && !stats_wait(sh, round)) lost = true;
  const float4 *v = sh.stats[round % kPlaces];
  RowStats r = {{v[0].x, 0.0f}, 0.0f, v[0].w};
  for (uint32_t i = 1; i < C; ++i) r.all.m = fmaxf(r.all.m, v[i].x);
  const float base = base_of(r.all.m);
  for (uint32_t i = 0; i < C; ++i) {
    r.all.s += v[i].y * exp2_sfu((v[i].x - base) * p.scale);
    r.parts += v[i].z;
  }
  if (lost) r.all.s = r.parts = __int_as_float(0x7fffffff);  // shows in loss and gradient
  return r;
}
// The lanes' sums together: referred to the largest reference first.
__device__ __forceinline__ MaxSum warp_join(MaxSum a, float scale) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = a.s * exp2_sfu((a.m - base_of(m)) * scale);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return {m, s};
}

// An entry warp of a block, for the even rows of its walk or the odd ones.
template <class E, bool kGrad>
__device__ __forceinline__ void entry_warp(const DistillParams &p, Shared &sh, float *arrays,
                                           uint32_t *seen, uint32_t parity, uint32_t rank,
                                           uint32_t C, uint32_t stride, int lane) {
  const E *logits = static_cast<const E *>(p.logits);
  Entries e;
  e.logp = arrays;
  e.p = e.logp + p.K;
  e.x = e.p + p.K;
  e.id = reinterpret_cast<int *>(e.x + p.K);
  int *next_id = e.id + p.K;
  for (uint32_t w = lane; kGrad && w < kSeen / 32; w += 32) seen[w] = 0;
  __syncwarp();
  auto nothing = [](uint32_t) {};
  bool lost = false;
  RowWalk walk(blockIdx.x / C, stride);
  uint32_t row = walk.learned(p, lane, nothing);
  if (parity) row = walk.learned(p, lane, nothing);
  Teacher teacher = {};
  if (row < p.N) teacher = load_teacher(p, row, lane, e.id, e.logp);
  for (uint32_t i = parity; row < p.N; i += 2) {
    uint32_t next = walk.learned(p, lane, nothing);
    next = walk.learned(p, lane, nothing);
    if (next < p.N) prefetch_entries(p, next, lane);
    const RowSlice<E> s(p, row, rank);
    const E *src = logits + (int64_t)row * p.logits_row;
    const int at = s.end_of(p, rank, lane);
    const float end = at >= 0 ? to_f32(src[at]) : kNegInf;  // this lane's logit at the row's ends
    const float weight = p.weight ? p.weight[row] : 1.0f;
    const EntrySums sums = teacher_entries<E>(p, src, s, rank, lane, e, teacher);
    if (lane == 0) barrier_expect(&sh.arrived[i % kPlaces], C * sizeof(float4));
    MaxSum mine = {end, end == kNegInf ? 0.0f : end == end ? 1.0f : end};
    named_wait(3 + parity);
    if (lane < row_threads() / 32)
      mine = join(mine, {sh.warp_stats[parity][lane].x, sh.warp_stats[parity][lane].y}, p.scale);
    mine = warp_join(mine, p.scale);
    if (lane < (int)C)
      send(remote_smem(&sh.stats[i % kPlaces][rank], lane),
           remote_smem(&sh.arrived[i % kPlaces], lane),
           make_float4(mine.m, mine.s, sums.part, sums.mass));
    // what the exchange does not wait for: on its way meanwhile
    __syncwarp();
    if (kGrad) join_repeated(p.K, lane, e, seen);
    if (next < p.N) teacher = load_teacher(p, next, lane, next_id, e.logp);
    const RowStats r = row_stats(p, sh, i, C, lost);
    if (rank == 0 && lane == 0) {
      float loss = r.parts + r.mass * fmaf(p.temp, logf(r.all.s), base_of(r.all.m) - sums.c);
      // a student without any logit above -inf gives the teacher's entries probability 0
      if (r.all.s == 0.0f) loss = -kNegInf;
      p.loss[row] = r.mass == 0.0f ? 0.0f : loss * p.temp;
    }
    if (kGrad) {
      const float w = weight * p.temp;
      const float f = r.all.s == 0.0f ? 0.0f : w * r.mass / r.all.s;
      E *dst = static_cast<E *>(p.dlogits) + (int64_t)row * p.dlogits_row;
      if (at >= 0)
        dst[at] = from_f32<E>(
            r.mass == 0.0f ? 0.0f : f * exp2_sfu((end - base_of(r.all.m)) * p.scale));
      __syncwarp();  // an entry there is another lane's
      named_wait(1 + parity);
      if (r.mass != 0.0f)
        for (uint32_t k = lane; k < p.K; k += 32)
          if (e.id[k] >= 0) {
            const float g = f * exp2_sfu((e.x[k] - base_of(r.all.m)) * p.scale);
            dst[e.id[k]] = from_f32<E>(fmaf(-w, e.p[k], g));
          }
      __syncwarp();
    }
    row = next;
    int *const ids = e.id;
    e.id = next_id, next_id = ids;
  }
}

// An unlearned row: no loss, no gradient.
template <class E, bool kGrad>
__device__ __noinline__ void unlearned(const DistillParams &p, uint32_t row, uint32_t rank,
                                       uint32_t nthr) {
  if (kGrad) {
    const RowSlice<E> s(p, row, rank);
    E *dst = static_cast<E *>(p.dlogits) + (int64_t)row * p.dlogits_row, *to = dst + s.from;
    const bool wide = ((uintptr_t)to & 15) == 0;
    for (uint32_t c = threadIdx.x; c < s.mine; c += nthr)
      store_chunk<E>(to + c * RowSlice<E>::kN, wide, make_uint4(0, 0, 0, 0));
    if (threadIdx.x < 32) {
      const int at = s.end_of(p, rank, threadIdx.x);
      if (at >= 0) dst[at] = from_f32<E>(0.0f);
    }
  }
  if (rank == 0 && threadIdx.x == 0) p.loss[row] = 0.0f;
}

template <class E, bool kGrad>
__global__ void __launch_bounds__(kMaxThreads, 3) distill_kernel(const DistillParams p) {
  constexpr int kN = 16 / sizeof(E);
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) Shared sh;
  const uint32_t rank = cluster_rank(), C = cluster_size();
  const uint32_t stride = gridDim.x / C;  // rows between two of a cluster
  // the last two warps have the entries, the others the rows
  const uint32_t tid = threadIdx.x, nthr = row_threads();
  const int lane = tid & 31, warp = tid >> 5;
  uint4 *slice = reinterpret_cast<uint4 *>(smem);
  if (tid == 0) {
    for (int i = 0; i < kPlaces; ++i) barrier_init(&sh.arrived[i]);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_arrive();  // the others' barriers are there before anything is sent
  cluster_wait();
  if (tid >= nthr) {
    const uint32_t parity = warp - nthr / 32;
    float *arrays = reinterpret_cast<float *>(smem + (size_t)p.slice * 16);
    uint32_t *seen = reinterpret_cast<uint32_t *>(arrays + kEntryWarps * 5 * p.K);
    entry_warp<E, kGrad>(p, sh, arrays + parity * 5 * p.K, seen + parity * (kSeen / 32),
                         parity, rank, C, stride, lane);
    return;
  }

  const E *logits = static_cast<const E *>(p.logits);
  E *dlogits = static_cast<E *>(p.dlogits);
  const Ch<2> scale = splat<2>(p.scale);
  bool lost = false;
  const uint32_t quarter = (p.slice + kGroups * nthr - 1) / (kGroups * nthr) * nthr;
  auto skip = [&](uint32_t row) { unlearned<E, kGrad>(p, row, rank, nthr); };
  RowWalk walk(blockIdx.x / C, stride);
  uint32_t row = walk.learned(p, lane, skip);
  RowSlice<E> slice_of(p, row < p.N ? row : 0, rank);  // of the row in hand
  if (row < p.N) {
    const RowSlice<E> s = slice_of;
    const E *from = logits + (int64_t)row * p.logits_row + s.from;
    uint32_t c = tid;
#pragma unroll 1
    for (uint32_t end = quarter; end <= kGroups * quarter; end += quarter) {
      for (; c < min(end, s.mine); c += nthr) copy_async<16>(slice + c, from + c * kN);
      copy_commit();
    }
  }
  for (uint32_t i = 0; row < p.N; ++i) {
    const uint32_t next = walk.learned(p, lane, skip);
    const float weight = kGrad && p.weight ? p.weight[row] : 1.0f;
    const uint32_t mine = slice_of.mine;
    const int at = slice_of.from;
    uint32_t mine_next = 0;
    const E *from = logits;
    if (next < p.N) {
      if (!p.same) slice_of = RowSlice<E>(p, next, rank);
      mine_next = slice_of.mine;
      from += (int64_t)next * p.logits_row + slice_of.from;
    }
    // The sum of this thread's chunks, as they arrive.
    MaxSum acc = {kNegInf, 0.0f};
    uint32_t c = tid;
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
      uint32_t next_c = c;
      const uint32_t end = (g + 1) * quarter, stop = min(end, mine);
      copy_wait_left(kGrad ? kGroups - 1 - g : kGroups - 1);
      if (g == 0) {  // the warp's first chunks give its reference
        float top = kNegInf;
        if (c < stop) top = chunk_max<E>(slice[c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        acc.m = top;
      }
#pragma unroll 2
      for (; c < stop; c += nthr) {
        const uint4 v = slice[c];
        float sum = chunk_sum<E>(v, -base_of(acc.m), scale);
        if (acc.m == kNegInf || !(sum < kFarAbove)) {  // or a NaN
          const float top = chunk_max<E>(v);
          if (top > acc.m) {
            acc.s *= exp2_sfu((acc.m - top) * p.scale);
            acc.m = top;
          }
          sum = chunk_sum<E>(v, -base_of(acc.m), scale);
        }
        acc.s += sum;
      }
      if (!kGrad) {  // nothing else wants the chunks
        for (; next_c < min(end, mine_next); next_c += nthr)
          copy_async<16>(slice + next_c, from + next_c * kN);
        copy_commit();
        c = next_c > c ? next_c : c;
      }
    }
    acc = warp_join(acc, p.scale);
    // the place was read when the round before the last had its statistics
    if (!kGrad && i >= 2 && !lost && !stats_wait(sh, i - 2)) lost = true;
    if (lane == 0) sh.warp_stats[i & 1][warp] = make_float2(acc.m, acc.s);
    __syncwarp();
    named_arrive(3 + (i & 1));
    if (kGrad) {
      const RowStats r = row_stats(p, sh, i, C, lost);
      acc = r.all;
      const float mass = r.mass;
      // no entry: nothing to learn, whatever the logits are
      const uint32_t keep = mass == 0.0f ? 0u : 0xffffffffu;
      const float w = weight * p.temp;
      const float f = acc.s == 0.0f ? 0.0f : w * mass / acc.s;  // of the exponentials
      const Ch<2> base = splat<2>(-base_of(acc.m)), by = splat<2>(f);
      E *to = dlogits + (int64_t)row * p.dlogits_row + at;
      const bool wide = ((uintptr_t)to & 15) == 0;
      c = tid;
#pragma unroll 1
      for (uint32_t end = quarter; end <= kGroups * quarter; end += quarter) {
        const uint32_t stop = min(end, max(mine, mine_next));
#pragma unroll 2
        for (; c < stop; c += nthr) {
          if (c < mine) {
            Ch<2> x[kN / 2];
            widen_chunk<E>(slice[c], x);
#pragma unroll
            for (int k = 0; k < kN / 2; ++k) {
              const Ch<2> y = (x[k] + base) * scale;
              x[k] = by * Ch<2>{exp2_sfu(y.v[0]), exp2_sfu(y.v[1])};
            }
            uint4 v = narrow_chunk<E>(x);
            v.x &= keep, v.y &= keep, v.z &= keep, v.w &= keep;
            store_chunk<E>(to + c * kN, wide, v);
          }
          if (c < mine_next) copy_async<16>(slice + c, from + c * kN);
        }
        copy_commit();
      }
      named_arrive(1 + (i & 1));
    }
    row = next;
  }
  copy_wait<0>();
}

// Bytes of a block's slice at most: three blocks share an SM below 72 KB, so that
// one's stores and copies run beside another's sums, two above.  (8192 rows of 297 KB,
// 151936 bfloat16: 707 us with four slices of 74 KB, 728 with eight of 37 KB.  Rows of 250
// KB: 566 us with four slices, 645 with eight, 790 with two of 125 KB.)
constexpr uint64_t kSliceBytes = 80 * 1024;

// Clusters that the GPU holds at a time (fewer than its room for their blocks,
// which have to lie in one part of it), asked once for a layout and device.
template <class... KArgs>
cudaError_t clusters_resident(void (*k)(KArgs...), const cudaLaunchConfig_t &cfg, int *n) {
  struct Known {
    const void *k;
    int device;
    unsigned cluster, threads;
    size_t smem;
    int n;
  };
  thread_local Known known[16];
  thread_local int count = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned cluster = cfg.attrs[0].val.clusterDim.x, threads = cfg.blockDim.x;
  for (int i = 0; i < (count < 16 ? count : 16); ++i) {
    const Known &c = known[i];
    if (c.k == (const void *)k && c.device == device && c.cluster == cluster &&
        c.threads == threads && c.smem == cfg.dynamicSmemBytes) {
      *n = c.n;
      return cudaSuccess;
    }
  }
  e = allow_shared_memory((const void *)k);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(n, k, &cfg);
  if (e == cudaSuccess && *n < 1) e = cudaErrorLaunchOutOfResources;
  if (e == cudaSuccess)
    known[count++ % 16] = {(const void *)k, device, cluster, threads, cfg.dynamicSmemBytes, *n};
  return e;
}

// Shared memory of a block: its slice, and two rows' entries.
size_t distill_smem(uint32_t slice, uint32_t K, bool grad) {
  return (size_t)slice * 16 + kEntryWarps * ((size_t)K * 20 + (grad ? kSeen / 8 : 0));
}

template <class E, bool kGrad>
cudaError_t launch(DistillParams &p, cudaStream_t st) {
  const uint32_t chunks = (uint32_t)((uint64_t)p.V * sizeof(E) / 16);  // of a row at most
  p.same = p.logits_row * sizeof(E) % 16 == 0;
  uint32_t C = 1;
  while (C < kMaxCluster && chunks > C * (kSliceBytes / 16)) C *= 2;
  p.slice = chunks ? (chunks + C - 1) / C : 1;
  const size_t smem = distill_smem(p.slice, p.K, kGrad);
  // A warp's work on a row beside its chunks is worth some 60 of them: eight warps
  // for the largest slices (64 KB, 8192 x 128256 bfloat16: 567 us, 637 with four), four for
  // smaller ones (37 KB, 8192 x 151936: 727 us with four, 815 with eight; 8 KB, 16384 x 4000
  // without and with the gradient: 56 and 92 us, 60 and 103 with two), two for the
  // smallest (2 KB, 16384 x 1000: 46 and 74 us, 48 and 76 with four).
  const unsigned threads =
      (p.slice >= 3500 ? 256 : p.slice >= 384 ? 128 : 64) + 32 * kEntryWarps;
  auto *k = distill_kernel<E, kGrad>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(C);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int resident = 0;
  cudaError_t e = clusters_resident(k, cfg, &resident);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  cfg.gridDim = dim3(C * (p.N < (uint32_t)resident ? p.N : (uint32_t)resident));
  ++launch_counter();
  e = cudaLaunchKernelEx(&cfg, k, (const DistillParams)p);
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
