// vec16.cuh -- 16 bytes of a row as fp32 values, and back (fp32: 4 values,
// bf16: 8; widening is exact, narrowing rounds to nearest even).
#pragma once

#include "common.cuh"

namespace twell {

// 16-byte load of a row that is read once: no L1 allocation, evict-first in
// L2.  Not the read-only path: the row may be the buffer that the same thread
// overwrites afterwards.
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p), "l"(gather_policy<L2_FIRST>())
               : "memory");
  return r;
}

// 16 bytes from global to shared memory, asynchronously, past L1.
__device__ __forceinline__ void copy16_async(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}
// The same with an L2 policy.
__device__ __forceinline__ void copy16_async(void *dst, const void *src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "l"(policy)
               : "memory");
}

template <typename E> constexpr int VEC16 = 16 / (int)sizeof(E);

__device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4], float *) {
  f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8], bf16 *) {
  f[0] = bf_lo(u.x); f[1] = bf_hi(u.x); f[2] = bf_lo(u.y); f[3] = bf_hi(u.y);
  f[4] = bf_lo(u.z); f[5] = bf_hi(u.z); f[6] = bf_lo(u.w); f[7] = bf_hi(u.w);
}
__device__ __forceinline__ uint4 pack16(const float (&f)[4], float *) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&f)[8], bf16 *) {
  return make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]),
                    pack_bf2(f[6], f[7]));
}

}  // namespace twell
