// Rows of a matrix moved in chunks of eight elements, whatever their alignment.
//
// A row is written in chunks that begin on a boundary of eight elements in memory, so
// that every store is whole; its first and last chunk may be in part outside the row.
// Where a row is read, the same eight columns may lie at any address: they are put
// together from the aligned 16-byte pieces that hold them.  A piece is read only where
// it holds an element that is wanted, so that nothing beyond the 16 bytes around an
// array's last element is touched.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "elem.cuh"

namespace nsk {

constexpr int kChunk = 8;  // elements

// Eight elements as they lie in memory.
template <class E>
struct Words {
  static constexpr int kN = 2 * (int)sizeof(E);
  uint32_t w[kN];
};

template <class E>
__device__ __forceinline__ void widen(const Words<E> &x, float (&v)[kChunk]) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = __uint_as_float(x.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i) {
      const Ch<2> p = widen_pair<E>(x.w[i]);
      v[2 * i] = p.v[0], v[2 * i + 1] = p.v[1];
    }
  }
}
template <class E>
__device__ __forceinline__ Words<E> narrow(const float (&v)[kChunk]) {
  Words<E> x;
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) x.w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i) x.w[i] = narrow_pair<E>(Ch<2>{v[2 * i], v[2 * i + 1]});
  }
  return x;
}

// Element i of the eight, and setting it (i known when the loop is unrolled).
template <class E>
__device__ __forceinline__ E element(const Words<E> &x, int i) {
  if constexpr (sizeof(E) == 4) {
    return __uint_as_float(x.w[i]);
  } else {
    const uint16_t h = (uint16_t)(x.w[i / 2] >> (16 * (i & 1)));
    return *reinterpret_cast<const E *>(&h);
  }
}
template <class E>
__device__ __forceinline__ void set_element(Words<E> &x, int i, E e) {
  if constexpr (sizeof(E) == 4) {
    x.w[i] = __float_as_uint(e);
  } else {
    const uint32_t h = *reinterpret_cast<const uint16_t *>(&e);
    x.w[i / 2] = (i & 1) ? (x.w[i / 2] & 0xffffu) | h << 16 : (x.w[i / 2] & 0xffff0000u) | h;
  }
}

__device__ __forceinline__ uint4 load16(const void *p) {
  return __ldg(static_cast<const uint4 *>(p));
}
// 32 bytes in one access, of a multiple of 32.
__device__ __forceinline__ void load32(const void *p, uint32_t (&w)[8]) {
  asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
        "=r"(w[7])
      : "l"(p));
}
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The eight elements at p, all of which are there.  kWhole: p is a multiple of their size.
template <class E, bool kWhole>
__device__ __forceinline__ Words<E> load_words(const E *p) {
  Words<E> x;
  const uint32_t off = kWhole ? 0 : (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
  if constexpr (sizeof(E) == 2) {
    if (off == 0) {
      const uint4 a = load16(p);
      x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
      return x;
    }
    const char *at = reinterpret_cast<const char *>(p) - off;
    const uint4 a = load16(at), b = load16(at + 16);
    uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) u[i] = u[i + 2];
    }
    if (off & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) u[i] = u[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x.w[i] = (off & 2) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
  } else {
    if (kWhole) {
      load32(p, x.w);
      return x;
    }
    const char *at = reinterpret_cast<const char *>(p) - off;
    const uint4 a = load16(at), b = load16(at + 16);
    uint32_t u[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0, 0, 0, 0};
    if (off) {
      const uint4 c = load16(at + 32);
      u[8] = c.x, u[9] = c.y, u[10] = c.z, u[11] = c.w;
    }
    if (off & 8) {
#pragma unroll
      for (int i = 0; i < 10; ++i) u[i] = u[i + 2];
    }
    if (off & 4) {
#pragma unroll
      for (int i = 0; i < 9; ++i) u[i] = u[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x.w[i] = u[i];
  }
  return x;
}

// Columns c to c + 7 of a row of D; those outside it are 0.
template <class E, bool kWhole>
__device__ __forceinline__ Words<E> load_columns(const E *row, int64_t c, int64_t D) {
  if constexpr (kWhole) {
    return load_words<E, true>(row + c);
  } else {
    if (c >= 0 && c + kChunk <= D) return load_words<E, false>(row + c);
    Words<E> x;
#pragma unroll
    for (int i = 0; i < Words<E>::kN; ++i) x.w[i] = 0;
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (c + i >= 0 && c + i < D) set_element(x, i, row[c + i]);
    return x;
  }
}

// The eight elements to a multiple of their size.
template <class E>
__device__ __forceinline__ void store_words(E *p, const Words<E> &x) {
  if constexpr (sizeof(E) == 2)
    *reinterpret_cast<uint4 *>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  else
    store32(p, x.w);
}
// Columns c to c + 7 of a row of D, where row + c is a multiple of their size.
template <class E, bool kWhole>
__device__ __forceinline__ void store_columns(E *row, int64_t c, int64_t D, const Words<E> &x) {
  if constexpr (kWhole) {
    store_words(row + c, x);
  } else {
    if (c >= 0 && c + kChunk <= D) {
      store_words(row + c, x);
      return;
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i)
      if (c + i >= 0 && c + i < D) row[c + i] = element(x, i);
  }
}

// Elements between the last boundary of eight elements and p: a row at p is written in
// chunks that begin at the columns -lead, 8 - lead, ...
template <class E, bool kWhole>
__device__ __forceinline__ int lead_of(const E *p) {
  if (kWhole) return 0;
  return (int)((uint32_t)reinterpret_cast<uintptr_t>(p) % (kChunk * sizeof(E)) / sizeof(E));
}

// Chunks that a row of D elements may touch.
__host__ __device__ __forceinline__ uint32_t chunks_of(uint32_t D, bool whole) {
  return whole ? D / kChunk : (uint32_t)(((uint64_t)D + 2 * kChunk - 2) / kChunk);
}

// Whether every row of D elements, `row` elements apart, begins and ends on a boundary.
inline bool whole_rows(const void *p, int64_t row, uint64_t D, uint64_t es) {
  return (reinterpret_cast<uintptr_t>(p) | (uint64_t)row * es | D * es) % (kChunk * es) == 0;
}

}  // namespace nsk
