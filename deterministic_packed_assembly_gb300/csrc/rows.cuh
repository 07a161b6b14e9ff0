// Rows of a matrix, eight columns a lane at a time, whatever their alignment.
//
// L lanes take 8 L neighbouring columns of a row (a span) in pieces of V elements, the
// widest that every row of the call begins at a multiple of: a lane's piece i begins at
// column (i L + lane) V of the span, so that neighbouring lanes move neighbouring pieces.  V
// = 8 moves 16 or 32 bytes at once; rows of an even number of elements are moved by
// pairs, odd ones by single elements.  (Putting aligned 16 bytes of odd rows together from
// two loads was measured once, on the first kernels: 100 columns in 16 bits, 6 experts: combine 144
// us; 1001 columns, 4 experts: 97.  Narrow pieces, with the distances known and whole spans without
// bounds, take 54 and 50; the other way was not measured on those.)
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "elem.cuh"

namespace nsk {

constexpr int kOct = 8;  // columns a lane has of a span

// A lane's eight columns as they lie in memory.
template <class E, int V>
struct Oct {
  static constexpr int kPieces = kOct / V;
  static constexpr int kBytes = V * (int)sizeof(E);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;  // of a piece
  uint32_t w[kPieces * kWords];
};

template <class E, int V>
__device__ __forceinline__ void clear(Oct<E, V> &x) {
#pragma unroll
  for (int i = 0; i < Oct<E, V>::kPieces * Oct<E, V>::kWords; ++i) x.w[i] = 0;
}

// Values widened before are forgotten: they are widened again, which costs less than the
// registers that keep them.
template <class E, int V>
__device__ __forceinline__ void forget(Oct<E, V> &x) {
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int i = 0; i < Oct<E, V>::kPieces * Oct<E, V>::kWords; ++i) asm volatile("" : "+r"(x.w[i]));
  }
}

template <int kBytes>
__device__ __forceinline__ void load_piece(const void *p, uint32_t *w) {
  if constexpr (kBytes == 32) {
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
          "=r"(w[7])
        : "l"(p));
  } else if constexpr (kBytes == 16) {
    const uint4 v = __ldg(static_cast<const uint4 *>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (kBytes == 8) {
    const uint2 v = __ldg(static_cast<const uint2 *>(p));
    w[0] = v.x, w[1] = v.y;
  } else if constexpr (kBytes == 4) {
    w[0] = __ldg(static_cast<const uint32_t *>(p));
  } else {
    w[0] = __ldg(static_cast<const uint16_t *>(p));
  }
}
template <int kBytes>
__device__ __forceinline__ void store_piece(void *p, const uint32_t *w) {
  if constexpr (kBytes == 32)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  else if constexpr (kBytes == 16)
    *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (kBytes == 8)
    *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  else if constexpr (kBytes == 4)
    *static_cast<uint32_t *>(p) = w[0];
  else
    *static_cast<uint16_t *>(p) = (uint16_t)w[0];
}

// Columns c, c + step, ... of a row of D, V of them each; what is beyond the row is left
// as it is (loads) or out (stores).  kAll: nothing is.  Bounds and distances that are not
// known cost more instructions than the moves themselves (20000 x 1001 bf16, 4 experts: combine
// 69 us, its gradient 125), so that whole spans of a warp go without.
template <bool kAll = false, class E, int V>
__device__ __forceinline__ void load_oct(Oct<E, V> &x, const E *row, uint32_t c, uint32_t step,
                                         uint32_t D) {
  using O = Oct<E, V>;
  const E *at = row + c;
#pragma unroll
  for (int i = 0; i < O::kPieces; ++i)
    if (kAll || c + i * step < D) load_piece<O::kBytes>(at + i * step, x.w + i * O::kWords);
}
template <bool kAll = false, class E, int V>
__device__ __forceinline__ void store_oct(E *row, uint32_t c, uint32_t step, uint32_t D,
                                          const Oct<E, V> &x) {
  using O = Oct<E, V>;
  E *at = row + c;
#pragma unroll
  for (int i = 0; i < O::kPieces; ++i)
    if (kAll || c + i * step < D) store_piece<O::kBytes>(at + i * step, x.w + i * O::kWords);
}
// Calls `body` with whether all of the columns up to `end` are in the row, known when it is
// compiled: for narrow pieces of a warp, whose bounds would take a test each (where a lane
// has one piece of a span, a second copy of the code costs more than its test).
template <int V, bool kWarp, class F>
__device__ __forceinline__ void by_all(uint32_t end, uint32_t D, F &&body) {
  if (V < kOct && kWarp && end <= D)
    body(std::integral_constant<bool, V < kOct && kWarp>{});
  else
    body(std::false_type{});
}

// The eight columns as pairs of floats, and back (each rounded once).
template <class E, int V>
__device__ __forceinline__ void widen(const Oct<E, V> &x, Ch<2> (&v)[kOct / 2]) {
#pragma unroll
  for (int i = 0; i < kOct / 2; ++i) {
    if constexpr (sizeof(E) == 4)
      v[i] = {__uint_as_float(x.w[2 * i]), __uint_as_float(x.w[2 * i + 1])};
    else if constexpr (V > 1)
      v[i] = widen_pair<E>(x.w[i]);
    else
      v[i] = widen_pair<E>(__byte_perm(x.w[2 * i], x.w[2 * i + 1], 0x5410));
  }
}
template <class E, int V>
__device__ __forceinline__ Oct<E, V> narrow(const Ch<2> (&v)[kOct / 2]) {
  Oct<E, V> x;
#pragma unroll
  for (int i = 0; i < kOct / 2; ++i) {
    if constexpr (sizeof(E) == 4) {
      x.w[2 * i] = __float_as_uint(v[i].v[0]), x.w[2 * i + 1] = __float_as_uint(v[i].v[1]);
    } else if constexpr (V > 1) {
      x.w[i] = narrow_pair<E>(v[i]);
    } else {
      const uint32_t p = narrow_pair<E>(v[i]);
      x.w[2 * i] = p, x.w[2 * i + 1] = p >> 16;
    }
  }
  return x;
}

// The widest pieces that an address, a row's length and the distance of rows are
// multiples of: 8, 2 or 1 elements.
inline int piece_of(const void *p, int64_t row, uint64_t D, uint64_t es) {
  const uint64_t all = reinterpret_cast<uintptr_t>(p) | (uint64_t)row * es | D * es;
  return all % (8 * es) == 0 ? 8 : all % (2 * es) == 0 ? 2 : 1;
}

// Lanes that take a row together: as few as have its columns, at most a warp; and how many
// spans it has.
inline uint32_t lanes_for(uint64_t D) {
  uint32_t lanes = 1;
  while (lanes < 32 && lanes * kOct < D) lanes *= 2;
  return lanes;
}
inline uint64_t spans_for(uint64_t D, uint32_t lanes) {
  return (D + lanes * kOct - 1) / (lanes * kOct);
}

}  // namespace nsk
