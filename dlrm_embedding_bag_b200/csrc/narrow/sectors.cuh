// Accesses of 32 bytes, a whole sector of memory each; pairs of f32 and of bf16 by one instruction.
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

// Two f32 as the pair that one instruction works on.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ float2 parts(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// (One by one: a sum of pairs is fused with a product in front of it, whatever it says.)
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const float2 x = parts(a), y = parts(b);
  return pair(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// 16 elements of T, as words, at p, which starts on 32 bytes, past the cache's order of use.
template <class T>
__device__ __forceinline__ void store_sector_words(T* p, const uint32_t (&w)[4 * sizeof(T)]) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(4 * sizeof(T)); i += 8)
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                     reinterpret_cast<uint32_t*>(p) + i),
                 "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                 "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                 : "memory");
}
template <class T>
__device__ __forceinline__ void store_sectors(T* p, const float* v) {
  uint32_t w[4 * sizeof(T)];
#pragma unroll
  for (int i = 0; i < static_cast<int>(4 * sizeof(T)); ++i)
    w[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : bf16_pair(v[2 * i], v[2 * i + 1]);
  store_sector_words(p, w);
}

}  // namespace dlrm
