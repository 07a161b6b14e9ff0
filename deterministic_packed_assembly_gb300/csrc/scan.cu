// The gated linear recurrence over packed rows, forward and backward.
//
//   a_t = sigmoid(f_t + bias), h_t = a_t p_t + (1 - a_t) z_t,
//   p_t = 0 where a sequence starts (pos 0), else h_{t-1}
//
// Each channel of each row is a chain of T steps.  A run of steps is the
// affine map h -> A h + H of the state before it, and two runs compose, so a
// chain is cut into segments of kSteps steps: a warp takes one segment of 32
// (or 64) channels, a lane one (or two) channels of it, all kSteps steps in
// registers; the block's eight warps take the eight segments of a tile, put
// their (A, H) in shared memory, and each one composes those before its own.
// Then it runs its steps again from the state it found (two multiply-adds a
// step) and writes them, so every input is read once.  Blocks walk along
// time; the loads of the next tile are in flight while a tile is computed.
// Where rows and channels are too few to fill the GPU, a cluster of up to
// eight blocks takes consecutive tiles and composes them through distributed
// shared memory: no block waits for another outside its cluster.
//
// A segment in which a sequence starts does not depend on the state before
// it.  Its A is -0.0: the sign says so (a product of gates has none), and the
// state before is then not used at all, so that a NaN of one document does
// not reach the next.
#include <cuda_runtime.h>

#include <cstdint>

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
static_assert(kTile == NS_SCAN_TILE, "states are saved at every tile");

struct ScanParams {
  const void *z, *f;
  int64_t z_row, z_time, f_row, f_time;
  const float *bias;
  const int32_t *pos, *doc;
  uint32_t B, T, D;
  uint32_t groups;  // of 32 lanes' channels
  uint32_t split;   // blocks of a cluster, along time
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

// a = sigmoid(x) and c = 1 - a = sigmoid(-x), neither by a subtraction that
// cancels: the small one of the two is exp(-|x|) / (1 + exp(-|x|)).
__device__ __forceinline__ void gate(float x, float &a, float &c) {
  const float e = exp2_sfu(-fabsf(x) * kLog2e);
  const float r = rcp_sfu(1.0f + e);
  const float small = e * r;
  const float large = 1.0f - small;  // the exact sum of both is 1
  const bool up = x >= 0.0f;
  a = up ? large : small;
  c = up ? small : large;
}

// The state after a run (A, H) that found the state h.
__device__ __forceinline__ float run_state(float A, float H, float h) {
  return __float_as_int(A) < 0 ? H : fmaf(A, h, H);
}

// One warp's segment of a tile as it lies in memory.
template <class E, int CH>
struct Segment {
  Vec<E, CH> z[kSteps], f[kSteps];
  int posv, docv;  // of step `lane`
  int n;           // steps inside the row
};

template <class E, int CH>
__device__ __forceinline__ void load_segment(const ScanParams &p, uint32_t b, int64_t t0,
                                             uint32_t c0, bool live, int lane,
                                             Segment<E, CH> &s) {
  const int64_t left = (int64_t)p.T - t0;
  s.n = left < 0 ? 0 : left > kSteps ? kSteps : (int)left;
  s.posv = 1;
  s.docv = 0;
  if (lane < s.n) {
    const int64_t i = (int64_t)b * p.T + t0 + lane;
    if (p.pos) s.posv = __ldg(p.pos + i);
    if (p.doc) s.docv = __ldg(p.doc + i);
  }
  const E *z = static_cast<const E *>(p.z) + (int64_t)b * p.z_row + t0 * p.z_time + c0;
  const E *f = static_cast<const E *>(p.f) + (int64_t)b * p.f_row + t0 * p.f_time + c0;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (live && i < s.n) {
      s.z[i] = *reinterpret_cast<const Vec<E, CH> *>(z + i * p.z_time);
      s.f[i] = *reinterpret_cast<const Vec<E, CH> *>(f + i * p.f_time);
    }
  }
}

// Bit i: a sequence starts at step i / step i is padding or past the row.
template <class E, int CH>
__device__ __forceinline__ void segment_flags(const Segment<E, CH> &s, int lane, uint32_t &reset,
                                              uint32_t &skip) {
  skip = __ballot_sync(0xffffffffu, lane >= s.n || s.docv < 0);
  reset = __ballot_sync(0xffffffffu, s.posv == 0) & ~skip;
}

// Gates and inputs of a segment; at skipped steps a = 1, c = 0, z = 0.
template <class E, int CH>
__device__ __forceinline__ void segment_gates(const Segment<E, CH> &s, const float (&bias)[CH],
                                              uint32_t skip, float (&a)[kSteps][CH],
                                              float (&c)[kSteps][CH], float (&z)[kSteps][CH]) {
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const bool out = (skip >> i) & 1u;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      gate(to_f32(s.f[i].v[k]) + bias[k], a[i][k], c[i][k]);
      z[i][k] = to_f32(s.z[i].v[k]);
      if (out) a[i][k] = 1.0f, c[i][k] = 0.0f, z[i][k] = 0.0f;
    }
  }
}

template <int CH>
__device__ __forceinline__ void load_channels(const float *src, int64_t off, bool live,
                                              float (&v)[CH]) {
#pragma unroll
  for (int k = 0; k < CH; ++k) v[k] = 0.0f;
  if (src && live) {
    const Vec<float, CH> x = *reinterpret_cast<const Vec<float, CH> *>(src + off);
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = x.v[k];
  }
}
template <int CH>
__device__ __forceinline__ void store_channels(float *dst, int64_t off, bool live,
                                               const float (&v)[CH]) {
  if (!dst || !live) return;
  Vec<float, CH> x;
#pragma unroll
  for (int k = 0; k < CH; ++k) x.v[k] = v[k];
  *reinterpret_cast<Vec<float, CH> *>(dst + off) = x;
}

// The runs of a tile's segments, or of a cluster's tiles, of 32 * CH channels.
template <int CH>
using Runs = float2[32 * CH];

template <class E, int CH, bool kCluster>
__global__ void __launch_bounds__(kThreads) scan_forward_kernel(const ScanParams p) {
  __shared__ Runs<CH> seg[2][kWarps];
  __shared__ Runs<CH> tile[kCluster ? 2 : 1][kCluster ? kMaxCluster : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = kCluster ? blockIdx.x % p.split : 0;
  const uint32_t unit = kCluster ? blockIdx.x / p.split : blockIdx.x;
  const uint32_t b = unit / p.groups, c0 = (unit % p.groups) * 32 * CH + lane * CH;
  const bool live = c0 < p.D;
  const int64_t nt = ((int64_t)p.T + kTile - 1) / kTile;
  if (kCluster) {  // the other blocks' shared memory is written to: they run
    cluster_arrive();
    cluster_wait();
  }
  float bias[CH], h[CH];
  load_channels<CH>(p.bias, c0, live, bias);
  load_channels<CH>(p.h0, (int64_t)b * p.D + c0, live, h);
  Segment<E, CH> next;
  load_segment<E, CH>(p, b, (int64_t)rank * kTile + warp * kSteps, c0, live, lane, next);
  int buf = 0;
  for (int64_t i = 0; i < nt; i += kCluster ? p.split : 1, buf ^= 1) {
    const int64_t j = i + rank;  // this block's tile: may lie past the last one
    const int64_t t0 = j * kTile + warp * kSteps;
    uint32_t reset, skip;
    float a[kSteps][CH], c[kSteps][CH], z[kSteps][CH];
    segment_flags<E, CH>(next, lane, reset, skip);
    segment_gates<E, CH>(next, bias, skip, a, c, z);
    const int n = next.n;
    load_segment<E, CH>(p, b, t0 + (int64_t)(kCluster ? p.split : 1) * kTile, c0, live, lane,
                        next);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float A = 1.0f, H = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bool start = (reset >> s) & 1u;
        H = fmaf(a[s][k], start ? 0.0f : H, c[s][k] * z[s][k]);
        A = start ? -0.0f : A * a[s][k];
      }
      seg[buf][warp][lane * CH + k] = make_float2(A, H);
    }
    __syncthreads();
    float in[CH];  // the state before this warp's segment
    if (kCluster) {
      float A[CH], H[CH], Aw[CH], Hw[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        A[k] = 1.0f, H[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w == warp) Aw[k] = A[k], Hw[k] = H[k];
          const float2 r = seg[buf][w][lane * CH + k];
          H[k] = run_state(r.x, r.y, H[k]);
          A[k] = __float_as_int(r.x) < 0 ? r.x : A[k] * r.x;
        }
      }
      if (warp < p.split) {  // warp w writes this tile's run into block w
        const uint32_t to = remote_smem(&tile[buf][rank][lane * CH], warp);
#pragma unroll
        for (int k = 0; k < CH; ++k)
          remote_store(to + k * sizeof(float2), make_float2(A[k], H[k]));
      }
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float mine = 0.0f;
        for (uint32_t r = 0; r < p.split; ++r) {
          if (r == rank) mine = h[k];
          const float2 x = tile[buf][r][lane * CH + k];
          h[k] = run_state(x.x, x.y, h[k]);
        }
        in[k] = run_state(Aw[k], Hw[k], mine);
      }
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w == warp) in[k] = h[k];
          const float2 r = seg[buf][w][lane * CH + k];
          h[k] = run_state(r.x, r.y, h[k]);
        }
      }
    }
    if (warp == 0 && j < nt)
      store_channels<CH>(p.states, ((int64_t)b * nt + j) * p.D + c0, live, in);
    E *y = static_cast<E *>(p.y) + ((int64_t)b * p.T + t0) * p.D + c0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      Vec<E, CH> out;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float before = (reset >> s) & 1u ? 0.0f : in[k];
        in[k] = fmaf(a[s][k], before, c[s][k] * z[s][k]);
        out.v[k] = from_f32<E>((skip >> s) & 1u ? 0.0f : in[k]);
      }
      if (live && s < n) *reinterpret_cast<Vec<E, CH> *>(y + (int64_t)s * p.D) = out;
    }
  }
  if (rank == 0 && warp == 0) store_channels<CH>(p.h_last, (int64_t)b * p.D + c0, live, h);
}

// Rows of at most kSteps steps: a thread takes a row's channels alone, one
// segment, no exchange.
template <class E, int CH>
__global__ void __launch_bounds__(kThreads) scan_forward_short_kernel(const ScanParams p) {
  const uint32_t per_row = (p.D + CH - 1) / CH;
  const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (uint64_t)p.B * per_row) return;
  const uint32_t b = (uint32_t)(i / per_row), c0 = (uint32_t)(i % per_row) * CH;
  float bias[CH], h[CH];
  load_channels<CH>(p.bias, c0, true, bias);
  load_channels<CH>(p.h0, (int64_t)b * p.D + c0, true, h);
  store_channels<CH>(p.states, (int64_t)b * p.D + c0, p.T > 0, h);
  const E *z = static_cast<const E *>(p.z) + (int64_t)b * p.z_row + c0;
  const E *f = static_cast<const E *>(p.f) + (int64_t)b * p.f_row + c0;
  E *y = static_cast<E *>(p.y) + (int64_t)b * p.T * p.D + c0;
#pragma unroll 2
  for (uint32_t t = 0; t < p.T; ++t) {
    const int64_t at = (int64_t)b * p.T + t;
    const bool start = p.pos && __ldg(p.pos + at) == 0, skip = p.doc && __ldg(p.doc + at) < 0;
    const Vec<E, CH> zv = *reinterpret_cast<const Vec<E, CH> *>(z + t * p.z_time);
    const Vec<E, CH> fv = *reinterpret_cast<const Vec<E, CH> *>(f + t * p.f_time);
    Vec<E, CH> out;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float a, c;
      gate(to_f32(fv.v[k]) + bias[k], a, c);
      const float to = fmaf(a, start ? 0.0f : h[k], c * to_f32(zv.v[k]));
      if (!skip) h[k] = to;
      out.v[k] = from_f32<E>(skip ? 0.0f : to);
    }
    *reinterpret_cast<Vec<E, CH> *>(y + (int64_t)t * p.D) = out;
  }
  store_channels<CH>(p.h_last, (int64_t)b * p.D + c0, true, h);
}

// The backward pass walks the tiles from the last one.  Inside a tile the
// states are run again from the saved one, forward in time, while
//   d_t = dy_t + u_t,  u_{t-1} = a_t d_t  (0 where a sequence starts)
// runs backward: both maps of a segment have the same A, and one exchange
// serves both.  Warp w takes the segment that is w-th from the tile's end.
template <class E, int CH, bool kCluster>
__global__ void __launch_bounds__(kThreads) scan_backward_kernel(const ScanParams p) {
  __shared__ Runs<CH> seg[2][kWarps];         // (A, H)
  __shared__ float seg_u[2][kWarps][32 * CH];  // U of the same segment
  __shared__ Runs<CH> tile[kCluster ? 2 : 1][kCluster ? kMaxCluster : 1];  // (A, U)
  __shared__ float sums[kWarps][32 * CH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = kCluster ? blockIdx.x % p.split : 0;
  const uint32_t unit = kCluster ? blockIdx.x / p.split : blockIdx.x;
  const uint32_t b = unit / p.groups, c0 = (unit % p.groups) * 32 * CH + lane * CH;
  const bool live = c0 < p.D;
  const int64_t nt = ((int64_t)p.T + kTile - 1) / kTile;
  const int64_t stride = kCluster ? p.split : 1;
  if (kCluster) {
    cluster_arrive();
    cluster_wait();
  }
  const E *dy = static_cast<const E *>(p.dy) + (int64_t)b * p.dy_row + c0;
  float bias[CH], u[CH], sum[CH];
  load_channels<CH>(p.bias, c0, live, bias);
  load_channels<CH>(p.dh_last, (int64_t)b * p.D + c0, live, u);
#pragma unroll
  for (int k = 0; k < CH; ++k) sum[k] = 0.0f;

  const int back = kWarps - 1 - warp;  // this warp's segment of a tile
  Segment<E, CH> next;
  Vec<E, CH> next_dy[kSteps];
  float next_h[CH];  // the saved state before the tile
  auto fetch = [&](int64_t j) {
    // a tile before the first one (past the last of the walk) has no steps
    const int64_t t0 = j < 0 ? (int64_t)p.T : j * kTile + back * kSteps;
    load_segment<E, CH>(p, b, t0, c0, live, lane, next);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (live && s < next.n)
        next_dy[s] = *reinterpret_cast<const Vec<E, CH> *>(dy + (t0 + s) * p.dy_time);
    load_channels<CH>(p.saved, ((int64_t)b * nt + j) * p.D + c0, live && j >= 0, next_h);
  };
  fetch(nt - 1 - rank);
  int buf = 0;
  for (int64_t i = 0; i < nt; i += stride, buf ^= 1) {
    const int64_t j = nt - 1 - i - rank;  // may be negative
    const int64_t t0 = j * kTile + back * kSteps;
    uint32_t reset, skip;
    float a[kSteps][CH], c[kSteps][CH], z[kSteps][CH], g[kSteps][CH], h[CH];
    segment_flags<E, CH>(next, lane, reset, skip);
    segment_gates<E, CH>(next, bias, skip, a, c, z);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int k = 0; k < CH; ++k) g[s][k] = (skip >> s) & 1u ? 0.0f : to_f32(next_dy[s].v[k]);
#pragma unroll
    for (int k = 0; k < CH; ++k) h[k] = next_h[k];
    const int n = next.n;
    fetch(j - stride);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float A = 1.0f, H = 0.0f, U = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bool start = (reset >> s) & 1u;
        H = fmaf(a[s][k], start ? 0.0f : H, c[s][k] * z[s][k]);
        A = start ? -0.0f : A * a[s][k];
      }
#pragma unroll
      for (int s = kSteps - 1; s >= 0; --s)
        U = (reset >> s) & 1u ? 0.0f : a[s][k] * (g[s][k] + U);
      seg[buf][warp][lane * CH + k] = make_float2(A, H);
      seg_u[buf][warp][lane * CH + k] = U;
    }
    __syncthreads();
    float ui[CH];  // u after this warp's segment, that is from its right
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      // the state before this segment: through the segments earlier in time
#pragma unroll
      for (int w = kWarps - 1; w > 0; --w) {
        const float2 r = seg[buf][w][lane * CH + k];
        if (w > warp) h[k] = run_state(r.x, r.y, h[k]);
      }
    }
    if (kCluster) {
      float A[CH], U[CH], Aw[CH], Uw[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        A[k] = 1.0f, U[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w == warp) Aw[k] = A[k], Uw[k] = U[k];
          const float ra = seg[buf][w][lane * CH + k].x;
          U[k] = run_state(ra, seg_u[buf][w][lane * CH + k], U[k]);
          A[k] = __float_as_int(ra) < 0 ? ra : A[k] * ra;
        }
      }
      if (warp < p.split) {
        const uint32_t to = remote_smem(&tile[buf][rank][lane * CH], warp);
#pragma unroll
        for (int k = 0; k < CH; ++k)
          remote_store(to + k * sizeof(float2), make_float2(A[k], U[k]));
      }
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float mine = 0.0f;
        for (uint32_t r = 0; r < p.split; ++r) {
          if (r == rank) mine = u[k];
          const float2 x = tile[buf][r][lane * CH + k];
          u[k] = run_state(x.x, x.y, u[k]);
        }
        ui[k] = run_state(Aw[k], Uw[k], mine);
      }
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w == warp) ui[k] = u[k];
          u[k] = run_state(seg[buf][w][lane * CH + k].x, seg_u[buf][w][lane * CH + k], u[k]);
        }
      }
    }
    // z becomes p_t - z_t, the rest of df's factors
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float before = (reset >> s) & 1u ? 0.0f : h[k];
        h[k] = fmaf(a[s][k], before, c[s][k] * z[s][k]);
        z[s][k] = before - z[s][k];
      }
    }
    const int64_t at = ((int64_t)b * p.T + t0) * p.D + c0;
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
      Vec<E, CH> oz, of;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const bool out = (skip >> s) & 1u;
        const float d = g[s][k] + ui[k], ad = a[s][k] * d;
        const float vz = out ? 0.0f : c[s][k] * d, vf = out ? 0.0f : c[s][k] * ad * z[s][k];
        ui[k] = (reset >> s) & 1u ? 0.0f : ad;
        oz.v[k] = from_f32<E>(vz);
        of.v[k] = from_f32<E>(vf);
        sum[k] += vf;
      }
      if (live && s < n) {
        *reinterpret_cast<Vec<E, CH> *>(static_cast<E *>(p.dz) + at + (int64_t)s * p.D) = oz;
        *reinterpret_cast<Vec<E, CH> *>(static_cast<E *>(p.df) + at + (int64_t)s * p.D) = of;
      }
    }
  }
  if (rank == 0 && warp == 0) store_channels<CH>(p.dh0, (int64_t)b * p.D + c0, live, u);
  if (p.partial) {
#pragma unroll
    for (int k = 0; k < CH; ++k) sums[warp][lane * CH + k] = sum[k];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
#pragma unroll
        for (int k = 0; k < CH; ++k) sum[k] += sums[w][lane * CH + k];
      store_channels<CH>(p.partial, ((int64_t)b * stride + rank) * p.D + c0, live, sum);
    }
  }
}

template <class E, int CH>
__global__ void __launch_bounds__(kThreads) scan_backward_short_kernel(const ScanParams p) {
  const uint32_t per_row = (p.D + CH - 1) / CH;
  const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (uint64_t)p.B * per_row) return;
  const uint32_t b = (uint32_t)(i / per_row), c0 = (uint32_t)(i % per_row) * CH;
  const int64_t bc = (int64_t)b * p.D + c0;
  float bias[CH], h[CH], u[CH], sum[CH];
  load_channels<CH>(p.bias, c0, true, bias);
  load_channels<CH>(p.saved, bc, p.T > 0, h);
  load_channels<CH>(p.dh_last, bc, true, u);
#pragma unroll
  for (int k = 0; k < CH; ++k) sum[k] = 0.0f;
  const E *z = static_cast<const E *>(p.z) + (int64_t)b * p.z_row + c0;
  const E *f = static_cast<const E *>(p.f) + (int64_t)b * p.f_row + c0;
  const E *dy = static_cast<const E *>(p.dy) + (int64_t)b * p.dy_row + c0;
  float a[kSteps][CH], c[kSteps][CH], q[kSteps][CH];  // q: p_t - z_t
  uint32_t start = 0, skip = 0;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s < (int)p.T) {
      const int64_t at = (int64_t)b * p.T + s;
      if (p.pos && __ldg(p.pos + at) == 0) start |= 1u << s;
      if (p.doc && __ldg(p.doc + at) < 0) skip |= 1u << s;
      const Vec<E, CH> zv = *reinterpret_cast<const Vec<E, CH> *>(z + s * p.z_time);
      const Vec<E, CH> fv = *reinterpret_cast<const Vec<E, CH> *>(f + s * p.f_time);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        gate(to_f32(fv.v[k]) + bias[k], a[s][k], c[s][k]);
        const float before = (start >> s) & 1u ? 0.0f : h[k], zk = to_f32(zv.v[k]);
        q[s][k] = before - zk;
        if (!((skip >> s) & 1u)) h[k] = fmaf(a[s][k], before, c[s][k] * zk);
      }
    }
  }
#pragma unroll
  for (int s = kSteps - 1; s >= 0; --s) {
    if (s < (int)p.T) {
      const bool out = (skip >> s) & 1u;
      const Vec<E, CH> gv = *reinterpret_cast<const Vec<E, CH> *>(dy + s * p.dy_time);
      Vec<E, CH> oz, of;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float d = to_f32(gv.v[k]) + u[k], ad = a[s][k] * d;
        const float vz = out ? 0.0f : c[s][k] * d, vf = out ? 0.0f : c[s][k] * ad * q[s][k];
        if (!out) u[k] = (start >> s) & 1u ? 0.0f : ad;
        oz.v[k] = from_f32<E>(vz);
        of.v[k] = from_f32<E>(vf);
        sum[k] += vf;
      }
      const int64_t at = ((int64_t)b * p.T + s) * p.D + c0;
      *reinterpret_cast<Vec<E, CH> *>(static_cast<E *>(p.dz) + at) = oz;
      *reinterpret_cast<Vec<E, CH> *>(static_cast<E *>(p.df) + at) = of;
    }
  }
  store_channels<CH>(p.dh0, bc, true, u);
  store_channels<CH>(p.partial, bc, true, sum);
}

// dbias[c] = the sum of the partial rows, in a fixed order: 32 channels a
// block, warp w the rows w, w + 8, ..., then the warps in order.
__global__ void __launch_bounds__(kThreads)
    scan_bias_kernel(const float *__restrict__ partial, uint64_t rows, uint32_t D, float *dbias) {
  pdl_wait_then_release();
  __shared__ float sums[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < D) {
#pragma unroll 8
    for (uint64_t r = warp; r < rows; r += kWarps) s += partial[r * D + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < D) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += sums[w][lane];
    dbias[c] = s;
  }
}

// Blocks along time: doubled while the grid holds fewer than three blocks a
// SM and every block of the cluster still has a tile.  The groups of 64
// channels count also where lanes take one channel each, so that the order of
// the sums depends on the sizes alone.
uint32_t split_of(uint32_t B, uint32_t T, uint32_t D) {
  const uint64_t units = (uint64_t)B * ((D + 63) / 64), nt = (T + (uint64_t)kTile - 1) / kTile;
  uint32_t s = 1;
  while (s < kMaxCluster && units * s < 456 && nt >= 2 * s) s *= 2;
  return s;
}

template <class... KArgs>
cudaError_t launch(void (*k)(KArgs...), uint64_t blocks, uint32_t cluster, cudaStream_t st,
                   const ScanParams &p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  ++launch_counter();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, p);
  const cudaError_t last = cudaGetLastError();
  return e != cudaSuccess ? e : last;
}

template <class E, int CH>
cudaError_t run_forward(ScanParams &p, cudaStream_t st) {
  if (p.T <= (uint32_t)kSteps) {
    const uint64_t n = (uint64_t)p.B * ((p.D + CH - 1) / CH);
    return launch(scan_forward_short_kernel<E, CH>, (n + kThreads - 1) / kThreads, 1, st, p);
  }
  p.groups = (p.D + 32 * CH - 1) / (32 * CH);
  p.split = split_of(p.B, p.T, p.D);
  const uint64_t blocks = (uint64_t)p.B * p.groups * p.split;
  return p.split > 1 ? launch(scan_forward_kernel<E, CH, true>, blocks, p.split, st, p)
                     : launch(scan_forward_kernel<E, CH, false>, blocks, 1, st, p);
}

template <class E, int CH>
cudaError_t run_backward(ScanParams &p, cudaStream_t st) {
  if (p.T <= (uint32_t)kSteps) {
    const uint64_t n = (uint64_t)p.B * ((p.D + CH - 1) / CH);
    return launch(scan_backward_short_kernel<E, CH>, (n + kThreads - 1) / kThreads, 1, st, p);
  }
  p.groups = (p.D + 32 * CH - 1) / (32 * CH);
  p.split = split_of(p.B, p.T, p.D);
  const uint64_t blocks = (uint64_t)p.B * p.groups * p.split;
  return p.split > 1 ? launch(scan_backward_kernel<E, CH, true>, blocks, p.split, st, p)
                     : launch(scan_backward_kernel<E, CH, false>, blocks, 1, st, p);
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
  const bool two = pairs(p, dtype == NS_F32 ? 4 : 2);
#define NSK_RUN(E, CH) \
  (kForward ? run_forward<E, CH>(p, st) : run_backward<E, CH>(p, st))
  switch (dtype) {
    case NS_F32: return two ? NSK_RUN(float, 2) : NSK_RUN(float, 1);
    case NS_BF16: return two ? NSK_RUN(__nv_bfloat16, 2) : NSK_RUN(__nv_bfloat16, 1);
    default: return two ? NSK_RUN(__half, 2) : NSK_RUN(__half, 1);
  }
#undef NSK_RUN
}

}  // namespace

cudaError_t launch_scan_forward(const ns_scan_inputs &in, const float *h0, void *y, float *h_last,
                                float *states, cudaStream_t st) {
  ScanParams p = params_of(in);
  p.h0 = h0, p.y = y, p.h_last = h_last, p.states = states;
  return run<true>(p, in.dtype, st);
}

uint64_t scan_partial_rows(uint32_t B, uint32_t T, uint32_t D) {
  return (uint64_t)B * (T <= (uint32_t)kSteps ? 1 : split_of(B, T, D));
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
  pdl_launch(scan_bias_kernel, dim3((in.D + 31) / 32), dim3(kThreads), 0, st,
             (const float *)partial, scan_partial_rows(in.B, in.T, in.D), in.D, dbias);
  return cudaGetLastError();
}

}  // namespace nsk
