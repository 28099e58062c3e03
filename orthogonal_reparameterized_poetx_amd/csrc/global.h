// Accesses through pointers that a kernel reads from a table in memory.  The
// compiler cannot see that such a pointer is a global one and would use flat
// accesses, which go through the LDS's address check and counter as well; the
// casts below say so.  No alignment beyond the element's is assumed by the
// 16-byte forms ending in _u.
#pragma once

#include "common.h"

namespace poetx {

#define POETX_GLOBAL __attribute__((address_space(1)))

template <typename T>
__device__ __forceinline__ T gld(const T* p) { return *(const POETX_GLOBAL T*)p; }
template <typename T>
__device__ __forceinline__ void gst(T* p, T v) { *(POETX_GLOBAL T*)p = v; }

// past the caches
template <typename T>
__device__ __forceinline__ T gld_nt(const void* p) { return __builtin_nontemporal_load((const POETX_GLOBAL T*)p); }
template <typename T>
__device__ __forceinline__ void gst_nt(void* p, T v) { __builtin_nontemporal_store(v, (POETX_GLOBAL T*)p); }

typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint4 gld16(const void* p) {
  return __builtin_bit_cast(uint4, *(const POETX_GLOBAL u32x4*)p);
}
__device__ __forceinline__ void gst16(void* p, uint4 v) {
  *(POETX_GLOBAL u32x4*)p = __builtin_bit_cast(u32x4, v);
}
__device__ __forceinline__ uint4 gld16_u(const void* p) {
  return __builtin_bit_cast(uint4, (u32x4)*(const POETX_GLOBAL u32x4_u*)p);
}
__device__ __forceinline__ void gst16_u(void* p, uint4 v) {
  *(POETX_GLOBAL u32x4_u*)p = (u32x4_u)__builtin_bit_cast(u32x4, v);
}

}  // namespace poetx
