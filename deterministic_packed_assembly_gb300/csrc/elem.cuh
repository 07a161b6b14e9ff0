// Element types and small device helpers of the training operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace nsk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// 2^x and 1/x by the special function unit (2 ulp and 1 ulp).  With them exp(x) is
// 2^(x log2 e), whose exponent is rounded: off by 2^-24 (1.3 |x| + 4) of itself, some 40
// units of a float's last place for a probability of e^-30, one or two for those that
// count.  Where each operator's sums are as near as that, the tests' bounds hold with room.
// An exponent carried in two floats takes four operations more a pair, and the kernels
// that stream logits have none to spare (distillation: 4093 x 50257 bfloat16 evaluated 103
// us in place of 77, 8192 x 128256 with the gradient 714 in place of 566).
__device__ __forceinline__ float exp2_sfu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_sfu(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---- pairs of floats ----------------------------------------------------------
// A lane's one or two channels, or values; two are computed by the packed
// instructions.  Each is rounded as written, never fused with another, so that the same
// formula has the same bits in every kernel.
template <int CH>
struct Ch;
template <>
struct Ch<1> {
  float v[1];
};
template <>
struct alignas(8) Ch<2> {
  float v[2];
};
__device__ __forceinline__ float2 pair(Ch<2> a) { return make_float2(a.v[0], a.v[1]); }
__device__ __forceinline__ Ch<1> fma(Ch<1> a, Ch<1> b, Ch<1> c) {
  return {fmaf(a.v[0], b.v[0], c.v[0])};
}
__device__ __forceinline__ Ch<2> fma(Ch<2> a, Ch<2> b, Ch<2> c) {
  const float2 r = __ffma2_rn(pair(a), pair(b), pair(c));
  return {r.x, r.y};
}
__device__ __forceinline__ Ch<1> operator*(Ch<1> a, Ch<1> b) { return {__fmul_rn(a.v[0], b.v[0])}; }
__device__ __forceinline__ Ch<2> operator*(Ch<2> a, Ch<2> b) {
  const float2 r = __fmul2_rn(pair(a), pair(b));
  return {r.x, r.y};
}
__device__ __forceinline__ Ch<1> operator+(Ch<1> a, Ch<1> b) { return {__fadd_rn(a.v[0], b.v[0])}; }
__device__ __forceinline__ Ch<2> operator+(Ch<2> a, Ch<2> b) {
  const float2 r = __fadd2_rn(pair(a), pair(b));
  return {r.x, r.y};
}
template <int CH>
__device__ __forceinline__ Ch<CH> splat(float x) {
  Ch<CH> r;
#pragma unroll
  for (int k = 0; k < CH; ++k) r.v[k] = x;
  return r;
}
// ---- asynchronous copies to shared memory ---------------------------------------
template <int kBytes>
__device__ __forceinline__ void copy_async(void *smem, const void *gmem) {
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem);
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(gmem), "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A pair of 16-bit elements in one register, and two floats.
template <class E>
__device__ __forceinline__ Ch<2> widen_pair(uint32_t x) {
  if constexpr (std::is_same<E, __nv_bfloat16>::value) {
    return {__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)};
  } else {
    const float2 v = __half22float2(*reinterpret_cast<__half2 *>(&x));
    return {v.x, v.y};
  }
}
template <class E>
__device__ __forceinline__ uint32_t narrow_pair(Ch<2> x) {
  if constexpr (std::is_same<E, __nv_bfloat16>::value) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x.v[0], x.v[1]);
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const __half2 v = __floats2half2_rn(x.v[0], x.v[1]);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}

// 16 bytes of elements as pairs of floats, and back.
template <class E>
__device__ __forceinline__ void widen_chunk(uint4 v, Ch<2> (&x)[8 / sizeof(E)]) {
  if constexpr (sizeof(E) == 4) {
    x[0] = {__uint_as_float(v.x), __uint_as_float(v.y)};
    x[1] = {__uint_as_float(v.z), __uint_as_float(v.w)};
  } else {
    x[0] = widen_pair<E>(v.x), x[1] = widen_pair<E>(v.y);
    x[2] = widen_pair<E>(v.z), x[3] = widen_pair<E>(v.w);
  }
}
template <class E>
__device__ __forceinline__ uint4 narrow_chunk(const Ch<2> (&x)[8 / sizeof(E)]) {
  if constexpr (sizeof(E) == 4)
    return make_uint4(__float_as_uint(x[0].v[0]), __float_as_uint(x[0].v[1]),
                      __float_as_uint(x[1].v[0]), __float_as_uint(x[1].v[1]));
  else
    return make_uint4(narrow_pair<E>(x[0]), narrow_pair<E>(x[1]), narrow_pair<E>(x[2]),
                      narrow_pair<E>(x[3]));
}

// ---- thread-block clusters --------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Arrive: this thread's shared-memory writes, to its own block and to the
// others, are visible to every thread of the cluster that waits after it.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// As cluster_arrive, with nothing to be seen: only that this thread got here.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
// The address, in block `rank` of the cluster, of this block's shared `p`.
__device__ __forceinline__ uint32_t remote_smem(const void *p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void remote_store(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y)
               : "memory");
}
__device__ __forceinline__ void remote_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// ---- barriers that asynchronous stores count down --------------------------------
__device__ __forceinline__ void barrier_init(uint64_t *bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(bar))
               : "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(bar)),
               "r"(bytes)
               : "memory");
}
// Wait for the phase of this parity; false if it has not come after about a second.
__device__ __forceinline__ bool barrier_wait(uint64_t *bar, uint32_t parity) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(bar);
  for (int i = 0; i < 100000; ++i) {  // each try suspends for some microseconds at most
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 10000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(at), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}
// Asynchronous store of 16 bytes to `to`, which counts them down at `bar` (both
// addresses of a block of the cluster).
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, float4 v) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(to),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
      : "memory");
}

}  // namespace nsk
