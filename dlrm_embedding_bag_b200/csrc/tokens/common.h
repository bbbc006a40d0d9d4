// What the kernels of libdlrm_tokens.so share: host-side bookkeeping, and
// loads and stores of the two element types through f32.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dlrm_sparse.h"

namespace dlrm {

// SMs of a B200. Grids and rules that need not follow the device at hand take this one:
// sizes of scratch must not depend on it, and a grid-stride loop does as well with it.
constexpr int kSms = 148;

// Records a failed CUDA call for dlrm_tokens_last_cuda_error(); DLRM_ERR_CUDA.
int cuda_fail(cudaError_t e);
// Counts kernel launches of this library (dlrm_tokens_launch_count).
void note_launch(int n = 1);
// SMs of the current device (0 and a recorded error if it cannot be asked).
int sm_count_current();
// cuTensorMapEncodeTiled, looked up once through the runtime (null if absent).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();

// A launch on `stream`; early: the kernel may be scheduled while the one before it
// is at work (programmatic dependent launch), else it waits for all before it.
template <class... P, class... A>
cudaError_t launch(void (*fn)(P...), dim3 grid, int threads, int smem, bool early,
                   cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

inline bool is_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline bool known_dtype(int d) { return d == DLRM_TABLE_F32 || d == DLRM_TABLE_BF16; }
inline int dtype_size(int d) { return d == DLRM_TABLE_BF16 ? 2 : 4; }
// Whether rows' base and pitch allow accesses of v elements (16 bytes at most each);
// that the rows' length is a multiple of v is the caller's to check.
inline bool rows_by(const void* p, int64_t ld, int elem, int v) {
  const int bytes = v * elem < 16 ? v * elem : 16;
  return is_aligned(p, bytes) && ld % v == 0;
}

// Elements of one 128-bit access.
template <class T>
constexpr int kVecOf = 16 / static_cast<int>(sizeof(T));

// VEC elements as they lie in memory: one, a pair, or a whole 128-bit access.
template <class T, int VEC>
struct RawOf {
  using type = uint4;
  static_assert(VEC == kVecOf<T>, "one 128-bit access");
};
template <class T>
struct RawOf<T, 1> {
  using type = T;
};
template <>
struct RawOf<float, 2> {
  using type = uint2;
};
template <>
struct RawOf<__nv_bfloat16, 2> {
  using type = uint32_t;
};
template <class T, int VEC>
using Raw = typename RawOf<T, VEC>::type;

// ... widened to f32 (a bf16 value is the upper half of an f32).
template <class T, int VEC>
__device__ __forceinline__ void widen(const Raw<T, VEC>& r, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = static_cast<float>(r);
  } else if constexpr (VEC == 2 && sizeof(T) == 4) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
  } else if constexpr (VEC == 2) {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xffff0000u);
  } else {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
}

template <class T, int VEC>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[VEC]) {
  widen<T, VEC>(*reinterpret_cast<const Raw<T, VEC>*>(p), v);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) |
         (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16);
}

// VEC values rounded to T (nearest even) at p, aligned to min(16, VEC *
// sizeof(T)) bytes. ONCE: nobody reads them soon; they leave L2 first, before what
// is read again.
template <class T, int VEC, bool ONCE = false>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[VEC]) {
  auto put = [](auto* at, auto value) {
    if constexpr (ONCE)
      __stcs(at, value);
    else
      *at = value;
  };
  if constexpr (VEC == 1) {
    if constexpr (sizeof(T) == 4)
      put(p, v[0]);
    else
      put(reinterpret_cast<unsigned short*>(p), __bfloat16_as_ushort(__float2bfloat16_rn(v[0])));
  } else if constexpr (VEC == 2) {
    if constexpr (sizeof(T) == 4)
      put(reinterpret_cast<float2*>(p), make_float2(v[0], v[1]));
    else
      put(reinterpret_cast<unsigned int*>(p), bf16x2_bits(v[0], v[1]));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      put(reinterpret_cast<float4*>(p + i), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
  } else if constexpr (VEC == 4) {
    put(reinterpret_cast<uint2*>(p), make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])));
  } else {
    static_assert(VEC == 8, "one 128-bit store");
    put(reinterpret_cast<uint4*>(p), make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                                                bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7])));
  }
}

}  // namespace dlrm
