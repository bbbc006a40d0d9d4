// Accesses of 32 bytes, a whole sector of memory each, and pairs of bf16 by one conversion.
#pragma once

#include <cstdint>

#include "tokens/common.h"

namespace dlrm {

// Two values rounded to bf16, the first in the lower half. (One instruction at the rate of
// other arithmetic; conversions one by one run at an eighth of it.)
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 bytes of T from v at p.
template <class T>
__device__ __forceinline__ void store_16_bytes(T* p, const float* v) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                              bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

__device__ __forceinline__ void load_32_bytes(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// 16 values at p, which starts on 32 bytes, past the cache's order of use.
template <class T>
__device__ __forceinline__ void store_sectors(T* p, const float* v) {
  constexpr int kWords = 4 * sizeof(T);
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    w[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : bf16_pair(v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < kWords; i += 8) {
    uint32_t* at = reinterpret_cast<uint32_t*>(p) + i;
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at),
                 "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                 "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                 : "memory");
  }
}

}  // namespace dlrm
