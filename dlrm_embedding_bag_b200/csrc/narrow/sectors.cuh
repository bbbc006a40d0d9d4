// Accesses of 32 bytes, a whole sector of memory each.
#pragma once

#include <cstdint>

#include "tokens/common.h"

namespace dlrm {

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
    w[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : bf16x2_bits(v[2 * i], v[2 * i + 1]);
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
