// The gated linear recurrence over packed rows, forward and backward.
//
//   a_t = sigmoid(f_t + bias), h_t = a_t p_t + (1 - a_t) z_t,
//   p_t = 0 where a sequence starts (pos 0), else h_{t-1}
//
// Each channel of each row is a chain of T steps.  A run of steps is the affine
// map h -> A h + H of the state before it, and two runs compose, so a chain is
// cut into segments of kSteps steps: a warp takes one segment of 64 channels (32
// of 32 bits), a lane two (one) of them, all kSteps steps in registers; the
// block's eight warps take the eight segments of a tile, put their runs in shared
// memory, and each one finds the state before its own.  Then it runs its steps
// again from that state and writes them: every input is read once.  Blocks walk
// along time, with asynchronous copies of the next two tiles in flight.  Where
// rows and channels are too few to fill the GPU, a cluster of up to eight blocks
// takes consecutive tiles and exchanges their runs through distributed shared
// memory.
//
// A segment in which a sequence starts does not depend on the state before it;
// that state is then not used at all (not even times 0), so that a NaN of one
// document does not reach the next.
//
// Forward 6 bytes an element move (16 bits), backward 10.  With two units on every SM
// nothing is used up: warps wait for arithmetic, shared memory and a tile's exchange (8 x
// 4096 x 2432 bfloat16: forward 95 us, 5.1 TB/s, DRAM 61 % and 58 % of the issue slots;
// backward 146 us, 5.5 TB/s, DRAM 66 % and 62 %).  Few units are bound by the latency of a
// round, 1.5 us in a block alone, 2 and 3 us in a cluster (1 x 32749 x 1001 floats: 130 and
// 196 us, 3.0 and 3.4 TB/s).
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

constexpr int kSteps = 8;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = kSteps * kWarps;
constexpr int kMaxCluster = 8;
constexpr int kShortSteps = NS_SCAN_TILE;  // rows up to this long can be a thread's alone
constexpr int kShortThreads = 128;
constexpr int kBiasWarps = 8;
static_assert(NS_SCAN_TILE % kSteps == 0, "states are saved at the start of a segment");
static_assert(kShortSteps <= kTile, "short rows are a tile, which is not split");
constexpr int kSaveEvery = NS_SCAN_TILE / kSteps;  // segments between two saved states

struct ScanParams {
  const void *z, *f;
  int64_t z_row, z_time, f_row, f_time;
  const float *bias;
  const int32_t *pos, *doc;
  uint32_t B, T, D;
  uint32_t groups;  // of 32 lanes' channels
  uint32_t split;   // blocks of a cluster, along time
  uint32_t first;   // the launch's first (row, group)
  uint32_t sums;    // partial sums of the bias's gradient that a row has
  int wide;         // bytes that rows are copied by: 16, 8, 4, or 2
  const void *z_end, *f_end, *dy_end;
  int step;         // steps from a warp's segment to its next one
  // and what that is in z, f, dy, in a contiguous [T][D] and in the saved states
  int64_t z_step, f_step, dy_step, out_step, state_step;
  // forward
  const float *h0;
  void *y;
  float *h_last;
  float *states;
  // backward
  const float *saved;
  const void *dy;
  int64_t dy_row, dy_time;
  const float *dh_last;
  void *dz, *df;
  float *partial, *dh0;
};

// a - b, as a + (-1) b: exact as a subtraction
template <int CH>
__device__ __forceinline__ Ch<CH> sub(Ch<CH> a, Ch<CH> b) {
  return fma(b, splat<CH>(-1.0f), a);
}
template <int CH>
__device__ __forceinline__ Ch<CH> pick(bool first, Ch<CH> a, Ch<CH> b) {
  Ch<CH> r;
#pragma unroll
  for (int k = 0; k < CH; ++k) r.v[k] = first ? a.v[k] : b.v[k];
  return r;
}
// A lane's channels of one step as they lie in memory: a pair of 16-bit ones in
// one register.  (A 32-bit lane takes one channel: its bytes are the same, and the
// registers of a second one are worth more than the packed instructions.)
template <class E, int CH>
struct RawOf;
template <class E>
struct RawOf<E, 1> {
  using type = E;
};
template <>
struct RawOf<__nv_bfloat16, 2> {
  using type = uint32_t;
};
template <>
struct RawOf<__half, 2> {
  using type = uint32_t;
};
template <class E, int CH>
using Raw = typename RawOf<E, CH>::type;

template <class E, int CH>
__device__ __forceinline__ Ch<CH> widen(Raw<E, CH> x) {
  if constexpr (CH == 1) {
    return {to_f32(x)};
  } else {
    return widen_pair<E>(x);
  }
}
template <class E, int CH>
__device__ __forceinline__ Raw<E, CH> narrow(Ch<CH> x) {
  if constexpr (CH == 1) {
    return from_f32<E>(x.v[0]);
  } else {
    return narrow_pair<E>(x);
  }
}
template <int CH>
__device__ __forceinline__ Ch<CH> load_channels(const float *src, int64_t off, bool live) {
  Ch<CH> r = splat<CH>(0.0f);
  if (src && live) r = *reinterpret_cast<const Ch<CH> *>(src + off);
  return r;
}
template <int CH>
__device__ __forceinline__ void store_channels(float *dst, int64_t off, bool live, Ch<CH> v) {
  if (dst && live) *reinterpret_cast<Ch<CH> *>(dst + off) = v;
}

// With x = f + bias and u = exp(x): c = 1 / (1 + u) = sigmoid(-x), and a = sigmoid(x) as u c
// where u < 1, else as 1 - c, each the form that keeps its digits there: a gate near 0
// is what is left of h0 and dh0 beside nothing else, and one near 1 is rounded once.
// Relative errors, with 2^-24 for 1: the exponent t is rounded, |x| + |bias| (log2 e itself
// is off by a quarter of |x|); 4 by 2^t and 2 by 1 / d (special function unit); 1 by
// the sum and 1 by the product.  (0 where c is below 2^-126.)  pb = bias log2 e.
template <int CH>
__device__ __forceinline__ void gate(Ch<CH> f, Ch<CH> pb, Ch<CH> &c, Ch<CH> &a) {
  const Ch<CH> t = fma(f, splat<CH>(kLog2e), pb);
  Ch<CH> u;
#pragma unroll
  for (int k = 0; k < CH; ++k) u.v[k] = exp2_sfu(t.v[k]);
  const Ch<CH> d = u + splat<CH>(1.0f);
#pragma unroll
  for (int k = 0; k < CH; ++k) c.v[k] = rcp_sfu(d.v[k]);
  const Ch<CH> low = u * c, high = sub(splat<CH>(1.0f), c);
#pragma unroll
  for (int k = 0; k < CH; ++k) a.v[k] = u.v[k] < 1.0f ? low.v[k] : high.v[k];
}

// A warp's ring of segments in shared memory, filled by asynchronous copies that
// run kRing - 1 tiles ahead: A arrays (z, f and, backward, dy) of kSteps rows.
// (Prefetched into registers instead, the backward kernel spilled at 128 of them
// and ran 16 warps an SM.)
constexpr int kRing = 3;
// Single 16-bit channels are copied as the 17 words that 32 of them may touch: their
// rows have room for 34, and begin at either half of the first word.
template <class E, int CH>
constexpr bool kHalves = sizeof(E) == 2 && CH == 1;
template <class E, int CH>
constexpr int kRowRoom = kHalves<E, CH> ? 34 : 32;
template <class E, int CH, int A>
struct alignas(16) Stage {
  Raw<E, CH> v[A][kSteps][kRowRoom<E, CH>];
};

// An array that is copied: where it lies, and its strides.
template <class E>
struct Source {
  const E *at;      // this lane's place in the segment that is copied next
  int64_t time;     // elements to the next step
  const E *begin, *end;  // of the array (kHalves)
};

// Copies of a segment's rows of 128 bytes by `p.wide` bytes a lane: 16 (kWide) where
// rows, strides and widths are multiples of them, a lane copying from every fourth
// row; 8; or 4.  Rows of 16-bit channels that begin at any 2 bytes are copied in the words
// they touch.
template <class E, int CH, bool kWide>
struct Copier {
  int row;        // the first row that this lane copies from, far out where it has none
  uint32_t into;  // byte of its row that it copies to

  // Sets this lane's place in an array whose segment's group starts at `group`.
  __device__ __forceinline__ Source<E> set(const ScanParams &p, const E *group, int64_t time,
                                           uint32_t width, int lane, const void *begin,
                                           const void *end) {
    if constexpr (kHalves<E, CH>) {
      row = lane <= 16 ? 0 : kSteps;
      into = lane * 4;
      return {group, time, static_cast<const E *>(begin), static_cast<const E *>(end)};
    } else {
      const int bytes = kWide ? 16 : p.wide, per_row = 128 / bytes, first = lane / per_row;
      into = lane % per_row * bytes;
      const uint32_t at = into / sizeof(E);
      row = at < width ? first : kSteps;
      return {group + first * time + at, time, nullptr, nullptr};
    }
  }
  template <int kBytes>
  __device__ __forceinline__ void rows(const Source<E> &from, int n, unsigned char *to,
                                       int lane) const {
    constexpr int kRows = kBytes / 4;
    to += lane / (32 / kRows) * 128 + into;
    if (kBytes == 4 && n == kSteps) {  // one branch in place of one a row
      if (row == kSteps) return;
      const E *at = from.at;
#pragma unroll
      for (int s = 0; s < kSteps; s += kRows, at += kRows * from.time)
        copy_async<kBytes>(to + s * 128, at);
      return;
    }
#pragma unroll
    for (int s = 0; s < kSteps; s += kRows)
      if (s + row < n) copy_async<kBytes>(to + s * 128, from.at + s * from.time);
  }
  // Copy steps [0, n) of the segment.
  __device__ __forceinline__ void copy(const ScanParams &p, const Source<E> &from, int n,
                                       uint32_t width, int lane,
                                       Raw<E, CH> (&dst)[kSteps][kRowRoom<E, CH>]) const {
    unsigned char *to = reinterpret_cast<unsigned char *>(dst);
    if constexpr (kHalves<E, CH>) {
      // words of rows of even and of odd steps: with an odd stride the halves alternate,
      // two steps on they are the same
      const uintptr_t even = (uintptr_t)from.at, odd = (uintptr_t)(from.at + from.time);
      const char *word[2] = {(const char *)(even & ~(uintptr_t)3) + into,
                             (const char *)(odd & ~(uintptr_t)3) + into};
      const int64_t two_steps = from.time * 4;
      const int channels = (int)min(width, 32u);
      const bool has[2] = {lane < ((int)(even & 2) / 2 + channels + 1) / 2,
                           lane < ((int)(odd & 2) / 2 + channels + 1) / 2};
      to += into;
      if (word[0] >= (const char *)from.begin && from.at + kSteps * from.time + 34 <= from.end) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          if (s + row < n && has[s % 2])
            copy_async<4>(to + s * sizeof(dst[0]), word[s % 2] + s / 2 * two_steps);
      } else {  // near the array's ends, whose elements may share a word with nothing
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if (s + row >= n || !has[s % 2]) continue;
          const E *w = reinterpret_cast<const E *>(word[s % 2] + s / 2 * two_steps);
          E *into_row = reinterpret_cast<E *>(to + s * sizeof(dst[0]));
          if (w >= from.begin) into_row[0] = w[0];
          if (w + 1 >= from.begin && w + 2 <= from.end) into_row[1] = w[1];
        }
      }
    } else {
      if (kWide) rows<16>(from, n, to, lane);
      else if (p.wide == 8) rows<8>(from, n, to, lane);
      else rows<4>(from, n, to, lane);
    }
  }
};

// Where a lane's channels lie in a row of a stage: in kHalves one element on where the
// row begins at a word's second half, which alternates with the step where the
// step's stride is odd.
template <class E, int CH, int A>
struct Places {
  int even[A], odd[A];
  __device__ __forceinline__ void set(int k, const E *group, int64_t time, int lane) {
    even[k] = odd[k] = lane;
    if constexpr (kHalves<E, CH>) {
      const int half = (int)((uintptr_t)group / 2 & 1);
      even[k] += half;
      odd[k] += (half + (int)time) & 1;
    }
  }
  __device__ __forceinline__ Ch<CH> read(const Stage<E, CH, A> &in, int k, int s, int lane) const {
    if constexpr (kHalves<E, CH>)
      return widen<E, CH>(in.v[k][s][s % 2 ? odd[k] : even[k]]);
    else
      return widen<E, CH>(in.v[k][s][lane]);
  }
};

// Steps inside the row from t on, at most kSteps.
__device__ __forceinline__ int steps_at(int T, int t) {
  return t < 0 ? 0 : min(max(T - t, 0), kSteps);
}

// Where sequences start and what is skipped (padding, steps past the row), for
// the segments that a warp takes one after the other, `step` apart: bits of four
// segments are read at once, a byte each, and four segments ahead.
struct Flags {
  int64_t at;  // of the first step of the next four segments, in this lane: in pos and doc
  int t;       // and in the row
  int posv, docv;
  uint32_t start, skip;

  __device__ __forceinline__ void load(const ScanParams &p, int step) {
    const bool in = t >= 0 && t < (int)p.T;
    posv = in && p.pos ? __ldg(p.pos + at) : 1;
    docv = in ? (p.doc ? __ldg(p.doc + at) : 0) : -1;
    t += 4 * step;
    at += 4 * step;
  }
  __device__ __forceinline__ void set(const ScanParams &p, uint32_t b, int t0, int step,
                                      int lane) {
    t = t0 + lane / kSteps * step + lane % kSteps;
    at = (int64_t)b * p.T + t;
    load(p, step);
  }
  // Before segment i of the walk.
  __device__ __forceinline__ void next(const ScanParams &p, int step, int i) {
    if ((i & 3) == 0) {
      skip = __ballot_sync(0xffffffffu, docv < 0);
      start = __ballot_sync(0xffffffffu, posv == 0) & ~skip;
      load(p, step);
    } else {
      skip >>= kSteps;
      start >>= kSteps;
    }
  }
};
static_assert(kSteps == 8, "a segment's flags are a byte");

// A run of steps maps the state h before it to A h + H, or, where a sequence
// starts inside (`cut`), to H alone.
template <int CH>
struct alignas(8 * CH) Run {
  Ch<CH> A, H;
};
template <int CH>
__device__ __forceinline__ Ch<CH> after(const Run<CH> &r, bool cut, Ch<CH> h) {
  return cut ? r.H : fma(r.A, h, r.H);
}
// A is a product of gates; K = 1 - A = c_0 a_1 a_2 ... + c_1 a_2 ... + ... is a sum of
// positive terms.  Near 1 each factor and product is rounded to a multiple of 2^-24 or
// 2^-25, the same way where the gates are alike, step after step, while K keeps the digits
// of the c.  So K is summed beside A over a quad, and what A is off by, e = (1 - A) - K, is
// added: A + A e is 1 - K, rounded once, but for e K, where A is near 1, and A, to its own
// digits, where it is near 0.  (A constant gate of f + bias = 10 is then off by 2^-24 each 32
// steps, not by 2^-25 each step and product.)
template <int CH>
__device__ __forceinline__ Ch<CH> factor(Ch<CH> A, Ch<CH> K) {
  return fma(A, sub(sub(splat<CH>(1.0f), A), K), A);
}
// Runs that warps or blocks exchange, N of them for every lane's channels.
template <int CH, int N>
struct Exchange {
  Run<CH> run[N][32];
  uint32_t cut[N];
};
// A tile's segments', with their K.
template <int CH>
struct Segments : Exchange<CH, kWarps> {
  Ch<CH> K[kWarps][32];
};

// A quad is four consecutive segments: NS_SCAN_TILE steps from a multiple of
// them, between two saved states.  The states at these boundaries are chained by
// the quads' runs, whichever blocks computed them, and the states inside follow
// from the one at the quad's start.  So a row's results do not depend on how
// its quads were shared out, nor on the other rows of the call.
constexpr int kQuad = kSaveEvery;
constexpr int kQuads = kWarps / kQuad;  // of a tile

template <int CH>
__device__ __forceinline__ Run<CH> quad_run(const Segments<CH> &x, int quad, int lane,
                                            uint32_t cuts) {
  Run<CH> all = x.run[quad * kQuad][lane];
  if (cuts == 0) {
    Ch<CH> K = x.K[quad * kQuad][lane];
#pragma unroll
    for (int k = 1; k < kQuad; ++k) {
      const Run<CH> r = x.run[quad * kQuad + k][lane];
      all.H = fma(r.A, all.H, r.H);
      all.A = all.A * r.A;
      K = fma(r.A, K, x.K[quad * kQuad + k][lane]);
    }
    all.A = factor(all.A, K);
  } else {
#pragma unroll
    for (int k = 1; k < kQuad; ++k) {
      const Run<CH> r = x.run[quad * kQuad + k][lane];
      all.H = after(r, x.cut[quad * kQuad + k] != 0, all.H);
    }
  }
  return all;
}
// Nonzero where a sequence starts in the quad.
template <int CH>
__device__ __forceinline__ uint32_t quad_cuts(const Segments<CH> &x, int quad) {
  const uint4 c = *reinterpret_cast<const uint4 *>(&x.cut[quad * kQuad]);
  return c.x | c.y | c.z | c.w;
}
// The state before this warp's segment, from the one before its quad.
template <int CH>
__device__ __forceinline__ Ch<CH> inside_quad(const Segments<CH> &x, int lane, int warp,
                                              uint32_t cuts, Ch<CH> h) {
  const int first = warp / kQuad * kQuad;
#pragma unroll
  for (int k = 0; k < kQuad - 1; ++k)
    if (first + k < warp)  // the same for the warp
      h = after(x.run[first + k][lane], cuts != 0 && x.cut[first + k] != 0, h);
  return h;
}

// In a block alone: the state before this warp's segment, from h before the tile, and after
// the segment's steps, which need nothing of it, h past the tile.  `mid` is the state before
// the tile's second quad for its warps, for the first one's still h.
static_assert(kQuads == 2, "the quads of a tile are written out");
template <int CH>
__device__ __forceinline__ Ch<CH> past_quad(const Segments<CH> &x, int quad, int lane, Ch<CH> h) {
  const uint32_t cuts = quad_cuts(x, quad);
  return after(quad_run(x, quad, lane, cuts), cuts != 0, h);
}
template <int CH>
__device__ __forceinline__ Ch<CH> pass_block(const Segments<CH> &x, int lane, int warp, Ch<CH> h,
                                             Ch<CH> &mid) {
  mid = warp < kQuad ? h : past_quad(x, 0, lane, h);  // the same for the warp
  return inside_quad(x, lane, warp, quad_cuts(x, warp / kQuad), mid);
}
template <int CH>
__device__ __forceinline__ Ch<CH> past_tile(const Segments<CH> &x, int lane, int warp, Ch<CH> mid) {
  if (warp < kQuad) mid = past_quad(x, 0, lane, mid);
  return past_quad(x, 1, lane, mid);
}

// In a cluster the blocks take consecutive tiles, and every quad's run
// is stored into every block, asynchronously: the stores themselves count down
// the barrier that the receiving block's warps wait at.  (A cluster barrier in
// its place has each warp wait for its earlier stores to global memory: a quarter
// of the stalls.)  A block sends round i + 1 when it has read round i, and has
// everything of round i, which the others sent after they had read round i - 1:
// two buffers do.
template <int CH>
struct Quads {
  Exchange<CH, kMaxCluster * kQuads> x;
  uint64_t arrived;  // an mbarrier
};

template <int CH>
__device__ __forceinline__ void send_run(uint32_t to, uint32_t bar, Run<CH> r) {
  if constexpr (CH == 2) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
        "[%5];" ::"r"(to),
        "f"(r.A.v[0]), "f"(r.A.v[1]), "f"(r.H.v[0]), "f"(r.H.v[1]), "r"(bar)
        : "memory");
  } else {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
            to),
        "f"(r.A.v[0]), "f"(r.H.v[0]), "r"(bar)
        : "memory");
  }
}
__device__ __forceinline__ void send_word(uint32_t to, uint32_t bar, uint32_t v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                   to),
               "r"(v), "r"(bar)
               : "memory");
}

template <int CH>
__device__ __forceinline__ void send_quad(const Segments<CH> &x, Quads<CH> &quads,
                                          uint32_t rank, uint32_t split, int lane, int warp) {
  const int quad = warp / kQuad;
  const uint32_t cuts = quad_cuts(x, quad);
  const Run<CH> all = quad_run(x, quad, lane, cuts);
  const uint32_t self = rank * kQuads + quad, count = split * kQuads;
  if (threadIdx.x == 0) barrier_expect(&quads.arrived, count * (32 * sizeof(Run<CH>) + 4));
  for (uint32_t to = warp % kQuad; to < split; to += kQuad) {
    const uint32_t bar = remote_smem(&quads.arrived, to);
    send_run<CH>(remote_smem(&quads.x.run[self][lane], to), bar, all);
    if (lane == 0) send_word(remote_smem(&quads.x.cut[self], to), bar, cuts);
  }
}
// The state before this warp's quad, and h moved on past the cluster's tiles.
template <int CH>
__device__ __forceinline__ Ch<CH> pass_cluster(const Quads<CH> &quads, uint64_t *arrived,
                                               uint32_t parity, bool &lost, uint32_t rank,
                                               uint32_t split, int lane, int warp, Ch<CH> &h) {
  const uint32_t self = rank * kQuads + warp / kQuad, count = split * kQuads;
  if (!lost && !barrier_wait(arrived, parity)) lost = true;
  const uint32_t any =
      __ballot_sync(0xffffffffu, (uint32_t)lane < count && quads.x.cut[lane] != 0);
  Ch<CH> mine = h;
  if (any == 0) {
#pragma unroll 4
    for (uint32_t q = 0; q < count; ++q) {
      if (q == self) mine = h;
      const Run<CH> r = quads.x.run[q][lane];
      h = fma(r.A, h, r.H);
    }
  } else {
    for (uint32_t q = 0; q < count; ++q) {
      if (q == self) mine = h;
      h = after(quads.x.run[q][lane], (any >> q) & 1u, h);
    }
  }
  if (lost) mine = h = splat<CH>(__int_as_float(0x7fffffff));  // shows in every output
  return mine;
}

// Blocks of an SM: 24 warps forward (80 registers), 16 backward (128).
constexpr int kForwardBlocks = 24 / kWarps, kBackwardBlocks = 16 / kWarps;
constexpr uint64_t kSMs = 152;

// Where a block works: a group of 32 lanes' channels of a row, and with others of
// its cluster every split-th tile.
struct Place {
  int lane, warp;
  uint32_t rank, b, cg, c0;
  bool live;
};
template <int CH, bool kCluster>
__device__ __forceinline__ Place place_of(const ScanParams &p) {
  Place at;
  at.lane = threadIdx.x & 31, at.warp = threadIdx.x >> 5;
  at.rank = kCluster ? blockIdx.x % p.split : 0;
  const uint32_t unit = p.first + (kCluster ? blockIdx.x / p.split : blockIdx.x);
  at.b = unit / p.groups, at.cg = (unit % p.groups) * 32 * CH, at.c0 = at.cg + at.lane * CH;
  at.live = at.c0 < p.D;
  return at;
}

template <int CH>
__device__ __forceinline__ void cluster_begin(Quads<CH> (&quads)[2]) {
  if (threadIdx.x == 0) {
    barrier_init(&quads[0].arrived);
    barrier_init(&quads[1].arrived);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_arrive();  // the others' barriers are there before anything is sent
  cluster_wait();
}

// ---- forward --------------------------------------------------------------------
// A segment's gates a and inputs c z, and K of its run; a = 1, c = 0 at skipped steps.
template <class E, int CH>
__device__ __forceinline__ void forward_gates(const Stage<E, CH, 2> &in,
                                              const Places<E, CH, 2> &at, int lane, Ch<CH> pb,
                                              uint32_t skip, Ch<CH> (&a)[kSteps],
                                              Ch<CH> (&cz)[kSteps], Ch<CH> &K) {
  const Ch<CH> zero = splat<CH>(0.0f);
  K = zero;
  if (skip == 0) {  // the same for the warp
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Ch<CH> c;
      gate<CH>(at.read(in, 1, s, lane), pb, c, a[s]);
      cz[s] = c * at.read(in, 0, s, lane);
      K = fma(a[s], K, c);
    }
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bool gone = (skip >> s) & 1u;
      Ch<CH> c;
      gate<CH>(at.read(in, 1, s, lane), pb, c, a[s]);
      a[s] = pick(gone, splat<CH>(1.0f), a[s]);
      cz[s] = pick(gone, zero, c * at.read(in, 0, s, lane));
      K = fma(a[s], K, pick(gone, zero, c));
    }
  }
}
template <int CH>
__device__ __forceinline__ Run<CH> forward_run(const Ch<CH> (&a)[kSteps],
                                               const Ch<CH> (&cz)[kSteps], Ch<CH> K,
                                               uint32_t start) {
  Run<CH> run = {a[0], cz[0]};
  if (start == 0) {
#pragma unroll
    for (int s = 1; s < kSteps; ++s) {
      run.H = fma(a[s], run.H, cz[s]);
      run.A = run.A * a[s];
    }
    run.A = factor(run.A, K);
  } else {  // A is not used
#pragma unroll
    for (int s = 1; s < kSteps; ++s)
      run.H = fma(a[s], pick((start >> s) & 1u, splat<CH>(0.0f), run.H), cz[s]);
  }
  return run;
}
// The segment's states from the one before it, into y.
template <class E, int CH>
__device__ __forceinline__ void forward_apply(const ScanParams &p, const Ch<CH> (&a)[kSteps],
                                              const Ch<CH> (&cz)[kSteps], Ch<CH> h, bool live,
                                              int left, uint32_t start, uint32_t skip, E *y) {
  if ((start | skip) == 0) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s, y += p.D) {
      h = fma(a[s], h, cz[s]);
      if (live) *reinterpret_cast<Raw<E, CH> *>(y) = narrow<E, CH>(h);
    }
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s, y += p.D) {
      h = fma(a[s], pick((start >> s) & 1u, splat<CH>(0.0f), h), cz[s]);
      if (live && s < left)
        *reinterpret_cast<Raw<E, CH> *>(y) =
            narrow<E, CH>(pick((skip >> s) & 1u, splat<CH>(0.0f), h));
    }
  }
}

// Blocks that each take a unit's whole row.
template <class E, int CH, bool kWide>
__global__ void __launch_bounds__(kThreads, kForwardBlocks)
    scan_forward_kernel(const ScanParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) Segments<CH> seg[2];
  const Place at = place_of<CH, false>(p);
  const int lane = at.lane, warp = at.warp;
  Stage<E, CH, 2> *ring = reinterpret_cast<Stage<E, CH, 2> *>(smem) + warp * kRing;
  release_dependents();
  const int T = (int)p.T, rounds = (T + kTile - 1) / kTile;
  int t = warp * kSteps;  // may lie past the row
  Copier<E, CH, kWide> copier;
  Places<E, CH, 2> places;
  const uint32_t width = p.D - at.cg;
  const E *group = static_cast<const E *>(p.z) + (int64_t)at.b * p.z_row + t * p.z_time + at.cg;
  Source<E> z_from = copier.set(p, group, p.z_time, width, lane, p.z, p.z_end);
  places.set(0, group, p.z_time, lane);
  group = static_cast<const E *>(p.f) + (int64_t)at.b * p.f_row + t * p.f_time + at.cg;
  Source<E> f_from = copier.set(p, group, p.f_time, width, lane, p.f, p.f_end);
  places.set(1, group, p.f_time, lane);
  auto fetch = [&](int at_step, Stage<E, CH, 2> &to) {
    const int n = steps_at(T, at_step);
    copier.copy(p, z_from, n, width, lane, to.v[0]);
    copier.copy(p, f_from, n, width, lane, to.v[1]);
    z_from.at += p.z_step, f_from.at += p.f_step;
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < kRing - 1; ++k) fetch(t + k * kTile, ring[k]);
  Flags flags;
  flags.set(p, at.b, t, kTile, lane);
  const Ch<CH> pb = load_channels<CH>(p.bias, at.c0, at.live) * splat<CH>(kLog2e);
  Ch<CH> h = load_channels<CH>(p.h0, (int64_t)at.b * p.D + at.c0, at.live);
  E *y = static_cast<E *>(p.y) + ((int64_t)at.b * p.T + t) * p.D + at.c0;
  int slot = 0;
  for (int i = 0; i < rounds; ++i, t += kTile) {
    __syncwarp();  // the slot that is filled now was read in the last round
    fetch(t + (kRing - 1) * kTile, ring[slot == 0 ? kRing - 1 : slot - 1]);
    flags.next(p, kTile, i);
    const uint32_t start = flags.start & 0xffu, skip = flags.skip & 0xffu;
    copy_wait<kRing - 1>();
    __syncwarp();
    Ch<CH> a[kSteps], cz[kSteps], K;
    forward_gates<E, CH>(ring[slot], places, lane, pb, skip, a, cz, K);
    slot = slot == kRing - 1 ? 0 : slot + 1;
    Segments<CH> &x = seg[i & 1];
    x.run[warp][lane] = forward_run<CH>(a, cz, K, start);
    x.K[warp][lane] = K;
    if (lane == 0) x.cut[warp] = start;
    __syncthreads();
    Ch<CH> mid;
    const Ch<CH> in = pass_block<CH>(x, lane, warp, h, mid);
    // the state before a quad is its first warp's to save
    if (p.states && warp % kQuad == 0)
      store_channels<CH>(p.states, ((int64_t)at.b * ((T + NS_SCAN_TILE - 1) / NS_SCAN_TILE) +
                                    t / NS_SCAN_TILE) * p.D + at.c0, at.live && t < T, in);
    forward_apply<E, CH>(p, a, cz, in, at.live, T - t, start, skip, y);
    h = past_tile<CH>(x, lane, warp, mid);
    y += p.out_step;
  }
  copy_wait<0>();
  if (warp == 0) store_channels<CH>(p.h_last, (int64_t)at.b * p.D + at.c0, at.live, h);
}

// Clusters of blocks, each with every split-th tile of a unit's row.  The runs of
// round i + 1 are computed and sent before the steps of round i are written, so
// that their way between the blocks lies beside this and the next round's runs.
// kAlone: two rounds' gates are in registers, for two blocks an SM, which is what grids
// of clusters alone hold anyway; else, beside blocks with whole rows, they are computed
// twice.
template <class E, int CH, bool kWide, bool kAlone>
__global__ void __launch_bounds__(kThreads, kAlone ? 2 : kForwardBlocks)
    scan_forward_cluster_kernel(const ScanParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) Segments<CH> seg[3];
  __shared__ __align__(16) unsigned char quads_mem[2 * sizeof(Quads<CH>)];
  Quads<CH>(&quads)[2] = *reinterpret_cast<Quads<CH>(*)[2]>(quads_mem);
  const Place at = place_of<CH, true>(p);
  const int lane = at.lane, warp = at.warp;
  Stage<E, CH, 2> *ring = reinterpret_cast<Stage<E, CH, 2> *>(smem) + warp * kRing;
  cluster_begin<CH>(quads);
  const int T = (int)p.T, rounds = (T + p.step - 1) / p.step;
  int t = (int)at.rank * kTile + warp * kSteps;  // may lie past the row
  Copier<E, CH, kWide> copier;
  Places<E, CH, 2> places;
  const uint32_t width = p.D - at.cg;
  const E *group = static_cast<const E *>(p.z) + (int64_t)at.b * p.z_row + t * p.z_time + at.cg;
  Source<E> z_from = copier.set(p, group, p.z_time, width, lane, p.z, p.z_end);
  places.set(0, group, p.z_time, lane);
  group = static_cast<const E *>(p.f) + (int64_t)at.b * p.f_row + t * p.f_time + at.cg;
  Source<E> f_from = copier.set(p, group, p.f_time, width, lane, p.f, p.f_end);
  places.set(1, group, p.f_time, lane);
  auto fetch = [&](int at_step, Stage<E, CH, 2> &to) {
    const int n = steps_at(T, at_step);
    copier.copy(p, z_from, n, width, lane, to.v[0]);
    copier.copy(p, f_from, n, width, lane, to.v[1]);
    z_from.at += p.z_step, f_from.at += p.f_step;
    copy_commit();
  };
  constexpr int kAhead = kAlone ? kRing - 1 : 1;  // tiles: a slot is read again where not alone
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(t + k * p.step, ring[k]);
  Flags flags;
  flags.set(p, at.b, t, p.step, lane);
  const Ch<CH> pb = load_channels<CH>(p.bias, at.c0, at.live) * splat<CH>(kLog2e);
  Ch<CH> h = load_channels<CH>(p.h0, (int64_t)at.b * p.D + at.c0, at.live);
  E *y = static_cast<E *>(p.y) + ((int64_t)at.b * p.T + t) * p.D + at.c0;
  bool lost = false;
  // What is left to do of a round whose runs are sent.
  struct Round {
    Ch<CH> a[kSteps], cz[kSteps];
    uint32_t start, skip;
  } now, next;
  // Round i's runs, its tile at step t_i.
  auto runs = [&](int i, int t_i, Round &r) {
    __syncwarp();
    fetch(t_i + kAhead * p.step, ring[(i + kAhead) % kRing]);
    flags.next(p, p.step, i);
    r.start = flags.start & 0xffu, r.skip = flags.skip & 0xffu;
    copy_wait<kAhead>();
    __syncwarp();
    Ch<CH> K;
    forward_gates<E, CH>(ring[i % kRing], places, lane, pb, r.skip, r.a, r.cz, K);
    Segments<CH> &x = seg[i % 3];
    x.run[warp][lane] = forward_run<CH>(r.a, r.cz, K, r.start);
    x.K[warp][lane] = K;
    if (lane == 0) x.cut[warp] = r.start;
    __syncthreads();
  };
  runs(0, t, now);
  send_quad<CH>(seg[0], quads[0], at.rank, p.split, lane, warp);
  for (int i = 0; i < rounds; ++i, t += p.step) {
    if (i + 1 < rounds) runs(i + 1, t + p.step, next);
    Quads<CH> &q = quads[i & 1];
    const Ch<CH> mine = pass_cluster<CH>(q, &q.arrived, (i >> 1) & 1, lost, at.rank, p.split, lane,
                                         warp, h);
    if (i + 1 < rounds) {
      __syncthreads();  // every warp has read round i
      send_quad<CH>(seg[(i + 1) % 3], quads[(i + 1) & 1], at.rank, p.split, lane, warp);
    }
    const Segments<CH> &x = seg[i % 3];
    const Ch<CH> in = inside_quad<CH>(x, lane, warp, quad_cuts(x, warp / kQuad), mine);
    if (p.states && warp % kQuad == 0)
      store_channels<CH>(p.states, ((int64_t)at.b * ((T + NS_SCAN_TILE - 1) / NS_SCAN_TILE) +
                                    t / NS_SCAN_TILE) * p.D + at.c0, at.live && t < T, in);
    if constexpr (!kAlone) {
      Ch<CH> K;
      forward_gates<E, CH>(ring[i % kRing], places, lane, pb, now.skip, now.a, now.cz, K);
    }
    forward_apply<E, CH>(p, now.a, now.cz, in, at.live, T - t, now.start, now.skip, y);
    now = next;
    y += p.out_step;
  }
  copy_wait<0>();
  if (p.h_last == p.h0) {  // the other blocks have taken their h0 into the states by here
    cluster_arrive();
    cluster_wait();
  }
  if (at.rank == 0 && warp == 0)
    store_channels<CH>(p.h_last, (int64_t)at.b * p.D + at.c0, at.live, h);
  pdl_wait();  // what waits for this launch also waits for the one before
}

// Rows of at most kShortSteps steps, which are one quad: a thread takes a row's
// channels alone, segment by segment, eight steps' loads in flight.  States at the
// segments' starts and the quad's end come from the segments' runs, as between warps:
// the results are the same bits as the blocks'.
template <class E, int CH>
struct ShortRow {
  Raw<E, CH> z[kSteps], f[kSteps];
  uint32_t start, skip;
  int n;
  // Steps [t0, t0 + kSteps) of the row, as many as it has.
  __device__ __forceinline__ void load(const ScanParams &p, uint32_t b, uint32_t c0, int t0) {
    n = min((int)p.T - t0, kSteps);
    const E *zp = static_cast<const E *>(p.z) + (int64_t)b * p.z_row + t0 * p.z_time + c0;
    const E *fp = static_cast<const E *>(p.f) + (int64_t)b * p.f_row + t0 * p.f_time + c0;
    const int64_t at = (int64_t)b * p.T + t0;
    start = skip = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s < n) {
        z[s] = *reinterpret_cast<const Raw<E, CH> *>(zp + s * p.z_time);
        f[s] = *reinterpret_cast<const Raw<E, CH> *>(fp + s * p.f_time);
        if (p.pos && __ldg(p.pos + at + s) == 0) start |= 1u << s;
        if (p.doc && __ldg(p.doc + at + s) < 0) skip |= 1u << s;
      }
    }
    start &= ~skip;  // padding starts nothing
  }
};
template <class E, int CH>
__global__ void __launch_bounds__(kShortThreads) scan_forward_short_kernel(const ScanParams p) {
  const uint32_t per_row = (p.D + CH - 1) / CH;
  const uint64_t i = (uint64_t)blockIdx.x * kShortThreads + threadIdx.x;
  if (i >= (uint64_t)p.B * per_row) return;
  const uint32_t b = (uint32_t)(i / per_row), c0 = (uint32_t)(i % per_row) * CH;
  const Ch<CH> pb = load_channels<CH>(p.bias, c0, true) * splat<CH>(kLog2e);
  Ch<CH> h = load_channels<CH>(p.h0, (int64_t)b * p.D + c0, true);
  store_channels<CH>(p.states, (int64_t)b * p.D + c0, p.T > 0, h);
  E *y = static_cast<E *>(p.y) + (int64_t)b * p.T * p.D + c0;
  ShortRow<E, CH> row;
  Run<CH> all = {splat<CH>(1.0f), splat<CH>(0.0f)};
  Ch<CH> all_K = splat<CH>(0.0f);
  bool cut = false;  // a sequence started
  const Ch<CH> first = h;
  for (int t0 = 0; t0 < (int)p.T; t0 += kSteps) {
    row.load(p, b, c0, t0);
    Run<CH> run = {splat<CH>(1.0f), splat<CH>(0.0f)};
    Ch<CH> in = h, K = splat<CH>(0.0f);
#pragma unroll
    for (int s = 0; s < kSteps; ++s, y += p.D) {
      if (s >= row.n) break;
      const bool gone = (row.skip >> s) & 1u, start = (row.start >> s) & 1u;
      Ch<CH> c, a;
      gate<CH>(widen<E, CH>(row.f[s]), pb, c, a);
      a = pick(gone, splat<CH>(1.0f), a);
      const Ch<CH> cz = pick(gone, splat<CH>(0.0f), c * widen<E, CH>(row.z[s]));
      in = fma(a, pick(start, splat<CH>(0.0f), in), cz);
      run.H = fma(a, pick(start, splat<CH>(0.0f), run.H), cz);
      run.A = run.A * a;
      K = fma(a, K, pick(gone, splat<CH>(0.0f), c));
      *reinterpret_cast<Raw<E, CH> *>(y) = narrow<E, CH>(pick(gone, splat<CH>(0.0f), in));
    }
    run.A = factor(run.A, K);
    h = after(run, row.start != 0, h);
    all.H = after(run, row.start != 0, all.H);
    all.A = all.A * run.A;
    all_K = fma(run.A, all_K, K);
    cut = cut || row.start != 0;
  }
  all.A = factor(all.A, all_K);
  store_channels<CH>(p.h_last, (int64_t)b * p.D + c0, true, after(all, cut, first));
}

// ---- backward -------------------------------------------------------------------
// The backward pass walks the tiles from the last one, and a warp's segments
// with them: warp w takes the segment that is w-th from the tile's end.
//   d_t = dy_t + u_t,  u_{t-1} = a_t d_t  (0 where a sequence starts: in the product's
//   place, which is a NaN where the gate is one)
// is a run in the other direction with the same A, exchanged as in the forward
// pass.  The states inside a quad are run again from the saved one before it,
// by the segments' forward runs, which are exchanged too.
//
// A segment's gates: a, c and q = da / dx; a = 1, c = q = 0 at
// skipped steps.
template <class E, int CH>
__device__ __forceinline__ void backward_gates(const Stage<E, CH, 3> &in,
                                               const Places<E, CH, 3> &at, int lane, Ch<CH> pb,
                                               uint32_t skip, Ch<CH> (&a)[kSteps],
                                               Ch<CH> (&c)[kSteps], Ch<CH> (&q)[kSteps]) {
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    gate<CH>(at.read(in, 1, s, lane), pb, c[s], a[s]);
    q[s] = a[s] * c[s];
  }
  if (skip) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bool gone = (skip >> s) & 1u;
      a[s] = pick(gone, splat<CH>(1.0f), a[s]);
      c[s] = pick(gone, splat<CH>(0.0f), c[s]);
      q[s] = pick(gone, splat<CH>(0.0f), q[s]);
    }
  }
}
// (A, U) of the segment, and H and K.
template <class E, int CH>
__device__ __forceinline__ Run<CH> backward_run(const Stage<E, CH, 3> &in,
                                                const Places<E, CH, 3> &at, int lane,
                                                const Ch<CH> (&a)[kSteps],
                                                const Ch<CH> (&c)[kSteps], uint32_t start,
                                                uint32_t skip, Ch<CH> &H, Ch<CH> &K) {
  const Ch<CH> zero = splat<CH>(0.0f);
  Run<CH> run = {splat<CH>(1.0f), zero};
  H = K = zero;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    run.A = run.A * a[s];
    K = fma(a[s], K, c[s]);
  }
  run.A = factor(run.A, K);
  if ((start | skip) == 0) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) H = fma(a[s], H, c[s] * at.read(in, 0, s, lane));
    Ch<CH> d = at.read(in, 2, kSteps - 1, lane);
#pragma unroll
    for (int s = kSteps - 2; s >= 0; --s) d = fma(a[s + 1], d, at.read(in, 2, s, lane));
    run.H = a[0] * d;
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const Ch<CH> cz = pick((skip >> s) & 1u, zero, c[s] * at.read(in, 0, s, lane));
      H = fma(a[s], pick((start >> s) & 1u, zero, H), cz);
    }
    Ch<CH> d = zero;
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
      const Ch<CH> g = pick((skip >> s) & 1u, zero, at.read(in, 2, s, lane));
      d = s == kSteps - 1 ? g : pick((start >> (s + 1)) & 1u, g, fma(a[s + 1], d, g));
    }
    run.H = pick(start & 1u, zero, a[0] * d);
  }
  return run;
}
// The state before this warp's segment, from the saved one before its quad:
// through the quad's earlier segments, which later warps hold.
template <int CH>
__device__ __forceinline__ Ch<CH> state_before(const Segments<CH> &x,
                                               const Ch<CH> (&ahead)[kWarps][32], int lane,
                                               int warp, Ch<CH> h) {
#pragma unroll
  for (int k = kQuad - 1; k > 0; --k) {
    if ((kWarps - 1 - warp) % kQuad >= k) {
      const Run<CH> r = {x.run[warp + k][lane].A, ahead[warp + k][lane]};
      h = after(r, x.cut[warp + k] != 0, h);
    }
  }
  return h;
}
// The segment's gradients, from the state before it and u after it.
template <class E, int CH>
__device__ __forceinline__ void backward_apply(const ScanParams &p, const Stage<E, CH, 3> &in,
                                               const Places<E, CH, 3> &at, int lane, const Ch<CH> (&a)[kSteps],
                                               const Ch<CH> (&c)[kSteps], Ch<CH> (&q)[kSteps],
                                               Ch<CH> h, Ch<CH> u, bool live, int left,
                                               uint32_t start, uint32_t skip, E *dz, E *df,
                                               Ch<CH> &sum) {
  const Ch<CH> zero = splat<CH>(0.0f);
  dz += (int64_t)(kSteps - 1) * p.D, df += (int64_t)(kSteps - 1) * p.D;
  if ((start | skip) == 0) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {  // q takes p_t - z_t in
      const Ch<CH> z = at.read(in, 0, s, lane);
      q[s] = q[s] * sub(h, z);
      h = fma(a[s], h, c[s] * z);
    }
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s, dz -= p.D, df -= p.D) {
      const Ch<CH> g = at.read(in, 2, s, lane);
      u = s == kSteps - 1 ? g + u : fma(a[s + 1], u, g);  // d_s
      const Ch<CH> d = u, vf = q[s] * d;
      sum = sum + vf;
      if (live) {
        *reinterpret_cast<Raw<E, CH> *>(dz) = narrow<E, CH>(c[s] * d);
        *reinterpret_cast<Raw<E, CH> *>(df) = narrow<E, CH>(vf);
      }
    }
  } else {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const Ch<CH> z = pick((skip >> s) & 1u, zero, at.read(in, 0, s, lane));
      const Ch<CH> before = pick((start >> s) & 1u, zero, h);
      q[s] = q[s] * sub(before, z);
      h = fma(a[s], before, c[s] * z);
    }
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s, dz -= p.D, df -= p.D) {
      const bool gone = (skip >> s) & 1u;
      const Ch<CH> g = pick(gone, zero, at.read(in, 2, s, lane));
      u = s == kSteps - 1 ? g + u : pick((start >> (s + 1)) & 1u, g, fma(a[s + 1], u, g));
      const Ch<CH> d = u, vf = pick(gone, zero, q[s] * d);
      sum = sum + vf;
      if (live && s < left) {
        *reinterpret_cast<Raw<E, CH> *>(dz) = narrow<E, CH>(pick(gone, zero, c[s] * d));
        *reinterpret_cast<Raw<E, CH> *>(df) = narrow<E, CH>(vf);
      }
    }
  }
}
// A block's part of the bias's gradient: `sum` over its warps.
template <int CH>
__device__ __forceinline__ void store_sums(const ScanParams &p, const Place &at,
                                           Ch<CH> (&room)[kWarps][32], Ch<CH> sum) {
  __syncthreads();
  room[at.warp][at.lane] = sum;
  __syncthreads();
  if (at.warp != 0) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) sum = sum + room[w][at.lane];
  float *to = p.partial + (int64_t)at.b * p.sums * p.D + at.c0;
  store_channels<CH>(to, (int64_t)at.rank * p.D, at.live, sum);
  for (uint32_t r = p.split + at.rank; r < p.sums; r += p.split)
    store_channels<CH>(to, (int64_t)r * p.D, at.live, splat<CH>(0.0f));
}

template <class E, int CH, bool kWide, bool kCluster>
__global__ void __launch_bounds__(kThreads, kBackwardBlocks)
    scan_backward_kernel(const ScanParams p) {
  constexpr int kSegs = kCluster ? 3 : 2;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) Segments<CH> seg[kSegs];  // (A, U)
  __shared__ Ch<CH> ahead[kSegs][kWarps][32];        // H of the same segments
  __shared__ __align__(16) unsigned char quads_mem[kCluster ? 2 * sizeof(Quads<CH>) : 16];
  Quads<CH>(&quads)[2] = *reinterpret_cast<Quads<CH>(*)[2]>(quads_mem);
  const Place at = place_of<CH, kCluster>(p);
  const int lane = at.lane, warp = at.warp;
  Stage<E, CH, 3> *ring = reinterpret_cast<Stage<E, CH, 3> *>(smem) + warp * kRing;
  if (kCluster) cluster_begin<CH>(quads);
  else release_dependents();
  const int T = (int)p.T, rounds = (T + p.step - 1) / p.step;
  const int back = kWarps - 1 - warp;  // this warp's segment of a tile
  // negative in a tile before the first one, past the end of the walk
  int t = ((T + kTile - 1) / kTile - 1 - (int)at.rank) * kTile + back * kSteps;
  Copier<E, CH, kWide> copier;
  Places<E, CH, 3> places;
  const uint32_t width = p.D - at.cg;
  const E *group = static_cast<const E *>(p.z) + (int64_t)at.b * p.z_row + t * p.z_time + at.cg;
  Source<E> z_from = copier.set(p, group, p.z_time, width, lane, p.z, p.z_end);
  places.set(0, group, p.z_time, lane);
  group = static_cast<const E *>(p.f) + (int64_t)at.b * p.f_row + t * p.f_time + at.cg;
  Source<E> f_from = copier.set(p, group, p.f_time, width, lane, p.f, p.f_end);
  places.set(1, group, p.f_time, lane);
  group = static_cast<const E *>(p.dy) + (int64_t)at.b * p.dy_row + t * p.dy_time + at.cg;
  Source<E> g_from = copier.set(p, group, p.dy_time, width, lane, p.dy, p.dy_end);
  places.set(2, group, p.dy_time, lane);
  auto fetch = [&](int at_step, Stage<E, CH, 3> &to) {
    const int n = steps_at(T, at_step);
    copier.copy(p, z_from, n, width, lane, to.v[0]);
    copier.copy(p, f_from, n, width, lane, to.v[1]);
    copier.copy(p, g_from, n, width, lane, to.v[2]);
    z_from.at -= p.z_step, f_from.at -= p.f_step, g_from.at -= p.dy_step;
    copy_commit();
  };
  // Copies run two tiles ahead in a block alone, one in a cluster, whose blocks
  // have two tiles in hand.
  constexpr int kAhead = kCluster ? 1 : kRing - 1;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(t - k * p.step, ring[k]);
  Flags flags;
  flags.set(p, at.b, t, -p.step, lane);
  // the saved state before the segment's quad
  const float *saved = p.saved + ((int64_t)at.b * ((T + NS_SCAN_TILE - 1) / NS_SCAN_TILE) +
                                  t / (int)NS_SCAN_TILE) * p.D + at.c0;
  Ch<CH> next_h = load_channels<CH>(saved, 0, at.live && t >= 0 && t < T);
  const Ch<CH> pb = load_channels<CH>(p.bias, at.c0, at.live) * splat<CH>(kLog2e);
  Ch<CH> u = load_channels<CH>(p.dh_last, (int64_t)at.b * p.D + at.c0, at.live);
  Ch<CH> sum = splat<CH>(0.0f);
  const int64_t out = ((int64_t)at.b * p.T + t) * p.D + at.c0;
  E *dz = static_cast<E *>(p.dz) + out, *df = static_cast<E *>(p.df) + out;
  bool lost = false;
  struct Round {
    Ch<CH> a[kSteps], c[kSteps], q[kSteps];
    uint32_t start, skip;
  };
  // Round i's runs, its tile at step t_i.
  auto runs = [&](int i, int t_i, int slot, int s, Round &r) {
    __syncwarp();
    fetch(t_i - kAhead * p.step, ring[slot + kAhead >= kRing ? slot + kAhead - kRing : slot + kAhead]);
    flags.next(p, -p.step, i);
    r.start = flags.start & 0xffu, r.skip = flags.skip & 0xffu;
    copy_wait<kAhead>();
    __syncwarp();
    backward_gates<E, CH>(ring[slot], places, lane, pb, r.skip, r.a, r.c, r.q);
    Ch<CH> H, K;
    seg[s].run[warp][lane] =
        backward_run<E, CH>(ring[slot], places, lane, r.a, r.c, r.start, r.skip, H, K);
    seg[s].K[warp][lane] = K;
    ahead[s][warp][lane] = H;
    if (lane == 0) seg[s].cut[warp] = r.start;
    __syncthreads();
  };
  auto take_state = [&](int t_i) {
    const Ch<CH> h = next_h;
    saved -= p.state_step;
    next_h = load_channels<CH>(saved, 0, at.live && t_i - p.step >= 0 && t_i - p.step < T);
    return h;
  };
  if constexpr (!kCluster) {
    int slot = 0;
    Round r;
    for (int i = 0; i < rounds; ++i, t -= p.step) {
      Ch<CH> h = take_state(t);
      runs(i, t, slot, i & 1, r);
      h = state_before<CH>(seg[i & 1], ahead[i & 1], lane, warp, h);
      Ch<CH> mid;
      const Ch<CH> ui = pass_block<CH>(seg[i & 1], lane, warp, u, mid);
      backward_apply<E, CH>(p, ring[slot], places, lane, r.a, r.c, r.q, h, ui, at.live, t < 0 ? 0 : T - t,
                            r.start, r.skip, dz, df, sum);
      u = past_tile<CH>(seg[i & 1], lane, warp, mid);
      dz -= p.out_step, df -= p.out_step;
      slot = slot == kRing - 1 ? 0 : slot + 1;
    }
  } else {  // as the forward pass's clusters
    int slot = 0, s = 0;
    Round now, next;
    runs(0, t, 0, 0, now);
    send_quad<CH>(seg[0], quads[0], at.rank, p.split, lane, warp);
    for (int i = 0; i < rounds; ++i, t -= p.step) {
      const int next_slot = slot == kRing - 1 ? 0 : slot + 1, next_s = s == 2 ? 0 : s + 1;
      if (i + 1 < rounds) runs(i + 1, t - p.step, next_slot, next_s, next);
      Quads<CH> &from = quads[i & 1];
      const Ch<CH> mine = pass_cluster<CH>(from, &from.arrived, (i >> 1) & 1, lost, at.rank,
                                           p.split, lane, warp, u);
      if (i + 1 < rounds) {
        __syncthreads();  // every warp has read round i
        send_quad<CH>(seg[next_s], quads[(i + 1) & 1], at.rank, p.split, lane, warp);
      }
      const Ch<CH> h = state_before<CH>(seg[s], ahead[s], lane, warp, take_state(t));
      const Ch<CH> ui = inside_quad<CH>(seg[s], lane, warp, quad_cuts(seg[s], warp / kQuad), mine);
      // two channels' gates of two rounds do not fit the registers: computed twice
      if constexpr (CH == 2)
        backward_gates<E, CH>(ring[slot], places, lane, pb, now.skip, now.a, now.c, now.q);
      backward_apply<E, CH>(p, ring[slot], places, lane, now.a, now.c, now.q, h, ui, at.live,
                            t < 0 ? 0 : T - t, now.start, now.skip, dz, df, sum);
      now = next;
      dz -= p.out_step, df -= p.out_step;
      slot = next_slot, s = next_s;
    }
  }
  copy_wait<0>();
  if (at.rank == 0 && warp == 0)
    store_channels<CH>(p.dh0, (int64_t)at.b * p.D + at.c0, at.live, u);
  if (p.partial) store_sums<CH>(p, at, ahead[0], sum);
  if (kCluster) pdl_wait();  // what waits for this launch also waits for the one before
}

// Backward, the states before every eight steps are kept, and those steps run again.
template <class E, int CH>
__global__ void __launch_bounds__(kShortThreads) scan_backward_short_kernel(const ScanParams p) {
  const uint32_t per_row = (p.D + CH - 1) / CH;
  const uint64_t i = (uint64_t)blockIdx.x * kShortThreads + threadIdx.x;
  if (i >= (uint64_t)p.B * per_row) return;
  const uint32_t b = (uint32_t)(i / per_row), c0 = (uint32_t)(i % per_row) * CH;
  const int64_t bc = (int64_t)b * p.D + c0;
  const Ch<CH> zero = splat<CH>(0.0f);
  const Ch<CH> pb = load_channels<CH>(p.bias, c0, true) * splat<CH>(kLog2e);
  Ch<CH> u = load_channels<CH>(p.dh_last, bc, true), sum = zero;
  Ch<CH> kept[kShortSteps / kSteps];
  kept[0] = load_channels<CH>(p.saved, bc, p.T > 0);
  ShortRow<E, CH> row;
#pragma unroll
  for (int k = 0; k + 1 < kShortSteps / kSteps; ++k) {
    kept[k + 1] = kept[k];
    if ((k + 1) * kSteps >= (int)p.T) continue;
    row.load(p, b, c0, k * kSteps);  // eight steps: more follow
    Run<CH> run = {splat<CH>(1.0f), zero};
    Ch<CH> K = zero;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bool gone = (row.skip >> s) & 1u;
      Ch<CH> c, a;
      gate<CH>(widen<E, CH>(row.f[s]), pb, c, a);
      a = pick(gone, splat<CH>(1.0f), a);
      const Ch<CH> cz = pick(gone, zero, c * widen<E, CH>(row.z[s]));
      run.H = fma(a, pick((row.start >> s) & 1u, zero, run.H), cz);
      run.A = run.A * a;
      K = fma(a, K, pick(gone, zero, c));
    }
    run.A = factor(run.A, K);
    kept[k + 1] = after(run, row.start != 0, kept[k]);
  }
  Run<CH> all = {splat<CH>(1.0f), zero};
  Ch<CH> all_K = zero;
  bool cut = false;
  const Ch<CH> last = u;
#pragma unroll
  for (int k = kShortSteps / kSteps - 1; k >= 0; --k) {
    const int t0 = k * kSteps;
    if (t0 >= (int)p.T) continue;
    row.load(p, b, c0, t0);
    const E *gp = static_cast<const E *>(p.dy) + (int64_t)b * p.dy_row + t0 * p.dy_time + c0;
    Raw<E, CH> g[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (s < row.n) g[s] = *reinterpret_cast<const Raw<E, CH> *>(gp + s * p.dy_time);
    Ch<CH> a[kSteps], c[kSteps], q[kSteps], h = kept[k];  // q: a c (p_t - z_t)
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      a[s] = splat<CH>(1.0f);
      c[s] = q[s] = zero;
      if (s < row.n && !((row.skip >> s) & 1u)) {
        gate<CH>(widen<E, CH>(row.f[s]), pb, c[s], a[s]);
        const Ch<CH> before = pick((row.start >> s) & 1u, zero, h);
        const Ch<CH> z = widen<E, CH>(row.z[s]);
        q[s] = a[s] * c[s] * sub(before, z);
        h = fma(a[s], before, c[s] * z);
      }
    }
    const int64_t at = ((int64_t)b * p.T + t0) * p.D + c0;
    E *dz = static_cast<E *>(p.dz) + at, *df = static_cast<E *>(p.df) + at;
    Run<CH> run = {splat<CH>(1.0f), zero};
    Ch<CH> ui = u;
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
      const bool have = s < row.n, after_start = s < kSteps - 1 && (row.start >> (s + 1)) & 1u;
      const bool gone = !have || ((row.skip >> s) & 1u);
      const Ch<CH> gs = gone ? zero : widen<E, CH>(g[s]);
      ui = s == kSteps - 1 ? gs + ui : pick(after_start, gs, fma(a[s + 1], ui, gs));
      const Ch<CH> d = ui, vf = pick(gone, zero, q[s] * d);
      run.H = s == kSteps - 1 ? gs : pick(after_start, gs, fma(a[s + 1], run.H, gs));
      sum = sum + vf;
      if (have) {
        *reinterpret_cast<Raw<E, CH> *>(dz + (int64_t)s * p.D) =
            narrow<E, CH>(pick(gone, zero, c[s] * d));
        *reinterpret_cast<Raw<E, CH> *>(df + (int64_t)s * p.D) = narrow<E, CH>(vf);
      }
    }
    run.H = pick(row.start & 1u, zero, a[0] * run.H);
    Ch<CH> K = zero;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      run.A = run.A * a[s];
      K = fma(a[s], K, c[s]);
    }
    run.A = factor(run.A, K);
    u = after(run, row.start != 0, u);
    all.H = after(run, row.start != 0, all.H);
    all.A = all.A * run.A;
    all_K = fma(run.A, all_K, K);
    cut = cut || row.start != 0;
  }
  all.A = factor(all.A, all_K);
  store_channels<CH>(p.dh0, bc, true, after(all, cut, last));
  store_channels<CH>(p.partial, bc, true, sum);
}

// dbias[c] = the sum of the partial rows, in a fixed order: 32 channels a
// block, warp w the rows w, w + 8, ..., then the warps in order.
__global__ void __launch_bounds__(32 * kBiasWarps)
    scan_bias_kernel(const float *__restrict__ partial, uint64_t rows, uint32_t D, float *dbias) {
  pdl_wait_then_release();
  __shared__ float sums[kBiasWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < D) {
#pragma unroll 8
    for (uint64_t r = warp; r < rows; r += kBiasWarps) s += partial[r * D + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < D) {
#pragma unroll
    for (int w = 1; w < kBiasWarps; ++w) s += sums[w][lane];
    dbias[c] = s;
  }
}

// How a call's units (a row's group of 64 channels, of 32 where a lane has single ones)
// are laid out: as many as give every SM the same number by a block each, the rest by
// clusters of blocks along time.
//
// Forward an SM has room for three blocks, and the clusters run in the room beside the
// others (8 rows of T = 4096, bfloat16: 320 units 107 us with the last 16 in clusters of
// four, 131 us by a block each, 112 us in clusters of eight; 160 units 78 us and 95 us;
// 376 units 117 us in clusters of two, 131 us by a block each; floats, 5 rows of T = 32749,
// 1024 channels: 442 us with the last 8 in clusters of four, 508 us all in clusters), but
// rows copied by 8 bytes or fewer a lane are slower there than in clusters alone (1001
// channels: 906 us and 602 us).  Backward two blocks fill an SM, and the rest comes after
// them (320 units 173 us, 230 us by a block each), unless it is more than a unit an SM (252
// units 147 us by a block each, 191 us in clusters).  Without others, and after them,
// clusters of four may be three blocks an SM (104 units backward 90 us, 100 us in
// clusters of two), those of eight two (44 units of T = 16384 forward 152 us, 134 us in
// clusters of four).
struct Layout {
  uint64_t whole;  // units taken by one block each
  uint32_t split;  // blocks for each of the others
};
Layout layout_of(uint64_t units, uint32_t T, bool forward, bool slow = false) {
  const uint64_t tiles = (T + (uint64_t)kTile - 1) / kTile;
  const uint64_t fill = forward ? kSMs : kBackwardBlocks * kSMs, whole = units / fill * fill;
  const uint64_t rest = units - whole;
  const bool beside = forward && whole / kSMs % kForwardBlocks != 0;
  uint32_t split = 1, most = beside ? kMaxCluster / 2 : kMaxCluster;
  auto fits = [&](uint32_t n) {
    const uint64_t blocks = beside ? 1 : n <= 4 ? 3 : 2;  // an SM
    return n <= most && rest * n <= blocks * kSMs && tiles >= n;
  };
  if (rest && rest <= kSMs)
    while (fits(2 * split)) split *= 2;
  if (slow && beside && whole == kSMs && split > 1) return {0, split};
  return {split == 1 ? units : whole, split};
}

uint64_t backward_units(uint32_t B, uint32_t D) { return (uint64_t)B * ((D + 63) / 64); }

template <class... KArgs>
cudaError_t launch(void (*k)(KArgs...), uint64_t blocks, unsigned threads, uint32_t cluster,
                   size_t smem, cudaStream_t st, const ScanParams &p, bool beside = false,
                   bool all = false) {
  if (smem > 0) {
    const cudaError_t e = allow_shared_memory((const void *)k, all);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  // the rest of a pass, beside the last blocks of its first launch
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? beside ? 2 : 1 : 0;
  ++launch_counter();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, p);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

// Whether a thread takes a row's channels alone: up to eight steps always.  Up to 32, where
// there are threads enough: they take T steps one after the other, the more at a time the
// more of them there are, blocks the same time for any T.  (Forward and backward in
// bfloat16, two channels a thread, us by threads and by blocks: T = 32, 49152 threads 36 and
// 37, 32768 32 and 26; T = 16, 12288 13.3 and 13.5, 8192 12.6 and 10.2; floats: T = 32, 65536
// 29 and 38, 32768 26 and 24.)  Single 16-bit channels always: by blocks they are copied in
// words with the half of another (T = 32, 8 x 1001: 18.5 and 19.3 us, 96 x 1001: 35 and 94).
bool short_rows(uint64_t threads, uint32_t T, bool halves) {
  return T <= (uint32_t)kSteps ||
         (T <= (uint32_t)kShortSteps && (halves || threads >= 48ull * T * T));
}

template <class E, int CH, bool kWide, bool kForward>
cudaError_t run_as(ScanParams &p, cudaStream_t st) {
  const uint64_t n = (uint64_t)p.B * ((p.D + CH - 1) / CH);
  if (short_rows(n, p.T, kHalves<E, CH>)) {
    return launch(kForward ? scan_forward_short_kernel<E, CH> : scan_backward_short_kernel<E, CH>,
                  (n + kShortThreads - 1) / kShortThreads, kShortThreads, 1, 0, st, p);
  }
  // Backward, where a lane has single channels, two groups count as a unit: the
  // workspace's size depends on the sizes alone.
  p.groups = (p.D + 32 * CH - 1) / (32 * CH);
  const uint64_t units = (uint64_t)p.B * p.groups;
  Layout l = layout_of(kForward ? units : backward_units(p.B, p.D), p.T, kForward,
                       CH == 1 && !kWide);
  if (!kForward && CH == 1) l.whole = l.split == 1 ? units : std::min(l.whole * 2, units);
  p.sums = l.split;
  const uint64_t whole = l.whole;
  const size_t smem = sizeof(Stage<E, CH, kForward ? 2 : 3>) * kRing * kWarps;
  auto part = [&](uint64_t first, uint64_t count, uint32_t split) {
    p.first = (uint32_t)first, p.split = split;
    p.step = (int)split * kTile;
    p.z_step = p.step * p.z_time, p.f_step = p.step * p.f_time, p.dy_step = p.step * p.dy_time;
    p.out_step = (int64_t)p.step * p.D, p.state_step = (int64_t)(p.step / (int)NS_SCAN_TILE) * p.D;
    return kForward
               ? launch(split == 1 ? scan_forward_kernel<E, CH, kWide>
                          : first > 0  ? scan_forward_cluster_kernel<E, CH, kWide, false>
                                       : scan_forward_cluster_kernel<E, CH, kWide, true>,
                        count * split, kThreads, split, smem, st, p, first > 0, kWide)
               : launch(split == 1 ? scan_backward_kernel<E, CH, kWide, false>
                                   : scan_backward_kernel<E, CH, kWide, true>,
                        count * split, kThreads, split, smem, st, p, first > 0, kWide);
  };
  if (whole) {
    const cudaError_t e = part(0, whole, 1);
    if (e != cudaSuccess || whole == units) return e;
  }
  return part(whole, units - whole, l.split);
}

// Two channels a lane need rows, strides and addresses of whole pairs.
bool pairs(const ScanParams &p, size_t es) {
  const uintptr_t e = (uintptr_t)p.z | (uintptr_t)p.f | (uintptr_t)p.y | (uintptr_t)p.dy |
                      (uintptr_t)p.dz | (uintptr_t)p.df;
  const uintptr_t s = (uintptr_t)p.bias | (uintptr_t)p.h0 | (uintptr_t)p.h_last |
                      (uintptr_t)p.states | (uintptr_t)p.saved | (uintptr_t)p.dh_last |
                      (uintptr_t)p.dh0 | (uintptr_t)p.partial;
  const int64_t st = p.z_row | p.z_time | p.f_row | p.f_time | p.dy_row | p.dy_time | p.D;
  return e % (2 * es) == 0 && s % 8 == 0 && st % 2 == 0;
}

// Bytes that rows can be copied by: 16, 8 or 4 where addresses, strides and widths
// are multiples of them, else 2.
int copied_by(const ScanParams &p, size_t es) {
  const int64_t st = p.z_row | p.z_time | p.f_row | p.f_time | p.dy_row | p.dy_time | p.D;
  const uint64_t all = (uint64_t)((uintptr_t)p.z | (uintptr_t)p.f | (uintptr_t)p.dy) |
                       (uint64_t)st * es;
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}
const void *end_of(const void *array, int64_t row, int64_t time, const ScanParams &p, size_t es) {
  if (!array || !p.B || !p.T) return array;
  return static_cast<const char *>(array) +
         ((int64_t)(p.B - 1) * row + (int64_t)(p.T - 1) * time + p.D) * (int64_t)es;
}

ScanParams params_of(const ns_scan_inputs &in) {
  ScanParams p = {};
  p.z = in.z, p.f = in.f;
  p.z_row = in.z_row, p.z_time = in.z_time, p.f_row = in.f_row, p.f_time = in.f_time;
  p.bias = in.bias, p.pos = in.pos, p.doc = in.doc;
  p.B = in.B, p.T = in.T, p.D = in.D;
  return p;
}

template <bool kForward>
cudaError_t run(ScanParams &p, int dtype, cudaStream_t st) {
  const size_t es = dtype == NS_F32 ? 4 : 2;
  const bool two = pairs(p, es);
  p.wide = copied_by(p, es);
  p.z_end = end_of(p.z, p.z_row, p.z_time, p, es);
  p.f_end = end_of(p.f, p.f_row, p.f_time, p, es);
  p.dy_end = end_of(p.dy, p.dy_row, p.dy_time, p, es);
  const bool wide = p.wide == 16;
#define NSK_PAIRS(E)                                       \
  (!two  ? run_as<E, 1, false, kForward>(p, st)            \
   : wide ? run_as<E, 2, true, kForward>(p, st)            \
          : run_as<E, 2, false, kForward>(p, st))
  switch (dtype) {
    case NS_F32:
      return wide ? run_as<float, 1, true, kForward>(p, st)
                  : run_as<float, 1, false, kForward>(p, st);
    case NS_BF16: return NSK_PAIRS(__nv_bfloat16);
    default: return NSK_PAIRS(__half);
  }
#undef NSK_PAIRS
}

}  // namespace

cudaError_t launch_scan_forward(const ns_scan_inputs &in, const float *h0, void *y, float *h_last,
                                float *states, cudaStream_t st) {
  ScanParams p = params_of(in);
  p.h0 = h0, p.y = y, p.h_last = h_last, p.states = states;
  return run<true>(p, in.dtype, st);
}

uint64_t scan_partial_rows(uint32_t B, uint32_t T, uint32_t D) {
  return (uint64_t)B * layout_of(backward_units(B, D), T, false).split;  // 1 for short rows
}

cudaError_t launch_scan_backward(const ns_scan_inputs &in, const float *states, const void *dy,
                                 int64_t dy_row, int64_t dy_time, const float *dh_last, void *dz,
                                 void *df, float *dbias, float *dh0, float *partial,
                                 cudaStream_t st) {
  ScanParams p = params_of(in);
  p.saved = states, p.dy = dy, p.dy_row = dy_row, p.dy_time = dy_time, p.dh_last = dh_last;
  p.dz = dz, p.df = df, p.dh0 = dh0, p.partial = dbias ? partial : nullptr;
  const cudaError_t e = in.B ? run<false>(p, in.dtype, st) : cudaSuccess;
  if (e != cudaSuccess || !dbias) return e;  // without rows dbias is 0
  ++launch_counter();
  pdl_launch(scan_bias_kernel, dim3((in.D + 31) / 32), dim3(32 * kBiasWarps), 0, st,
             (const float *)partial, scan_partial_rows(in.B, in.T, in.D), in.D, dbias);
  return cudaGetLastError();
}

}  // namespace nsk
