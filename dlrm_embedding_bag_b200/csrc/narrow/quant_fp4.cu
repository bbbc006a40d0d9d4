// Rows rounded to 4-bit floating point with a scale for each 32 elements, and back
// (declared in dlrm_fp4.h).
//
// Bound by reading the rows (f32: 4 bytes an element against 0.53 written). The
// scale's exponent is the largest magnitude's own, carried up where its mantissa is above
// 7/4: an integer addition to its bits. Products with powers of two are exact (where they
// do not vanish, and then the code is 0), so a code is one rounding of its element.
//
// Two forms. Where rows start on 16 bytes a thread takes half a block, 16 elements, in
// accesses of 16 or 32 bytes, and a block's two threads exchange their maxima. Elsewhere a
// lane takes one column of several blocks, so that a warp still reads neighbours.
#include <algorithm>
#include <climits>

#include "fp4_common.cuh"
#include "tokens/common.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr uint32_t kInfBits = 0x7f800000u;

struct QuantArgs {
  const void* x;
  uint8_t* q;
  uint8_t* scale;
  int64_t ldx, ldq, block_tiles;
  int M, K;
  int rows, blocks;  // with the scales' padding: multiples of 128 and of 4
  Divisor by;        // a row's blocks, or kUnits of them
};

// A block's scale byte from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int e = static_cast<int>((top + 0x1fffffu) >> 23) - 2;
  return top >= kInfBits ? 255u : static_cast<uint32_t>(max(e, 0));
}

// 2^(127 - E), a normal number for every E that a finite block gets.
__device__ __forceinline__ float inverse_of(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Two elements as codes, the first in the low half of the byte.
__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b16 %0, {b, 0};\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void load_32_bytes(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// BYTES (16 or 32) at a time.
template <int BYTES, int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t part[8];
    const char* at = static_cast<const char*>(p) + 4 * i;
    if constexpr (BYTES == 32) {
      load_32_bytes(at, part);
    } else {
      const uint4 a = reinterpret_cast<const uint4*>(at)[0], b = reinterpret_cast<const uint4*>(at)[1];
      part[0] = a.x, part[1] = a.y, part[2] = a.z, part[3] = a.w;
      part[4] = b.x, part[5] = b.y, part[6] = b.z, part[7] = b.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) w[i + k] = part[k];
  }
}

// Half a block a thread.
template <class T, int BYTES>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kWords = 16 * sizeof(T) / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t pair = i >> 1;
  const int row = static_cast<int>(a.by.of(pair));
  const int block = static_cast<int>(pair - static_cast<int64_t>(row) * a.blocks);
  const int half = static_cast<int>(i & 1);
  const int c = block * 32 + half * 16;
  const bool live = row < a.M && c < a.K;
  uint32_t w[kWords] = {};
  const T* x = static_cast<const T*>(a.x) + row * a.ldx + c;
  if (live && c + 16 <= a.K) {
    load_words<BYTES>(x, w);
  } else if (live) {
    for (int e = 0; e < 16; ++e)
      if (c + e < a.K) {
        // (an index that the compiler knows would keep w in registers; this is one
        // thread of a row)
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            if (k == e) w[k] = __float_as_uint(x[e]);
        } else {
          const uint32_t b = reinterpret_cast<const uint16_t*>(x)[e];
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            if (k == e / 2) w[k] |= b << (16 * (e & 1));
        }
      }
  }
  uint32_t top = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) top = max(top, w[k] & 0x7fffffffu);
  } else {
    uint32_t two = 0;
#pragma unroll
    for (int k = 0; k < kWords; ++k) two = __vmaxu2(two, w[k] & 0x7fff7fffu);
    top = max(two & 0xffff0000u, two << 16);
  }
  top = max(top, __shfl_xor_sync(kFull, top, 1));
  const uint32_t byte = scale_byte(top);
  const float inv = byte == 255u ? 0.f : inverse_of(byte);
  if (row < a.rows && half == 0) a.scale[fp4_scale_at(a.block_tiles, row, block)] = byte;
  if (!live) return;
  uint32_t out[2] = {};
  if (byte != 255u) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float lo, hi;
      if constexpr (sizeof(T) == 4) {
        lo = __uint_as_float(w[2 * k]), hi = __uint_as_float(w[2 * k + 1]);
      } else {
        lo = __uint_as_float(w[k] << 16), hi = __uint_as_float(w[k] & 0xffff0000u);
      }
      out[k / 4] |= codes_of(lo * inv, hi * inv) << (8 * (k % 4));
    }
  }
  uint8_t* q = a.q + row * a.ldq + c / 2;
  if (c + 16 <= a.K && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
    *reinterpret_cast<uint2*>(q) = make_uint2(out[0], out[1]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + 2 * k < a.K) q[k] = static_cast<uint8_t>(out[k / 4] >> (8 * (k % 4)));
  }
}

// A column a lane, kUnits blocks of a row a warp.
constexpr int kUnits = 4;

template <class T>
__global__ void __launch_bounds__(kThreads) quantize_by_lanes_kernel(const QuantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int units = a.blocks / kUnits;  // blocks is a multiple of 4
  const int row = static_cast<int>(a.by.of(unit));
  const int block0 = static_cast<int>(unit - static_cast<int64_t>(row) * units) * kUnits;
  if (row >= a.rows) return;
  float v[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int c = (block0 + u) * 32 + lane;
    v[u] = 0.f;
    if (row < a.M && c < a.K)
      v[u] = static_cast<float>((static_cast<const T*>(a.x) + row * a.ldx)[c]);
  }
  uint32_t scales = 0;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const uint32_t top = __reduce_max_sync(kFull, __float_as_uint(fabsf(v[u])));
    const uint32_t byte = scale_byte(top);
    scales |= byte << (8 * u);
    const float mine = byte == 255u ? 0.f : v[u] * inverse_of(byte);
    const float next = __shfl_down_sync(kFull, mine, 1);
    const int c = (block0 + u) * 32 + lane;
    if ((lane & 1) == 0 && row < a.M && c < a.K)
      (a.q + row * a.ldq)[c / 2] = static_cast<uint8_t>(byte == 255u ? 0u : codes_of(mine, next));
  }
  if (lane == 0)
    *reinterpret_cast<uint32_t*>(a.scale + fp4_scale_at(a.block_tiles, row, block0)) = scales;
}

// Back to values: 16 elements a thread, or one where rows do not start on 16 bytes.
struct DequantArgs {
  const uint8_t* q;
  const uint8_t* scale;
  void* y;
  int64_t ldq, ldy, block_tiles;
  int M, K, groups;  // of 16 (or 1) elements in a row
  Divisor by;        // groups
};

__device__ __forceinline__ float value_of(uint32_t code, float scale) {
  // the sign, then exponent and mantissa as an f32's, whose bias 2^126 corrects
  return __uint_as_float((code & 8u) << 28 | (code & 7u) << 22) * 0x1p126f * scale;
}

template <class T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = a.by.of(i);
  if (row >= a.M) return;
  const int c = static_cast<int>(i - row * a.groups) * 16;
  const float scale = fp4_scale_value(a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), c / 32)]);
  const uint2 w = *reinterpret_cast<const uint2*>(a.q + row * a.ldq + c / 2);
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = value_of(((e < 8 ? w.x : w.y) >> (4 * (e % 8))) & 15u, scale);
  T* y = static_cast<T*>(a.y) + row * a.ldy + c;
  constexpr int V = kVecOf<T>;
#pragma unroll
  for (int e = 0; e < 16; e += V) store_f32<T, V>(y + e, *reinterpret_cast<const float(*)[V]>(v + e));
}

template <class T>
__global__ void __launch_bounds__(kThreads) dequantize_one_kernel(const DequantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = a.by.of(i);
  if (row >= a.M) return;
  const int c = static_cast<int>(i - row * a.groups);
  const float v[1] = {
      value_of((a.q[row * a.ldq + c / 2] >> (4 * (c & 1))) & 15u,
               fp4_scale_value(a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), c / 32)]))};
  store_f32<T, 1>(static_cast<T*>(a.y) + row * a.ldy + c, v);
}

constexpr int64_t kMost = INT_MAX - 1024;
// Largest M * K (rounded up to whole scale tiles): no grid leaves 2^31 blocks and no
// quotient its Divisor's range. (180 GB hold 2^37 elements of bf16.)
constexpr int64_t kMostElements = int64_t{1} << 38;

bool fits(int64_t M, int64_t K) {
  return (M + 127) / 128 * fp4_block_tiles(K) <= kMostElements / (128 * 128) && M * K < kMostElements;
}

template <class T>
cudaError_t run_quantize(QuantArgs a, cudaStream_t s) {
  const int64_t pitch = a.ldx * static_cast<int64_t>(sizeof(T));
  const int64_t threads = static_cast<int64_t>(a.rows) * a.blocks * 2;
  if (is_aligned(a.x, 16) && (pitch % 16 == 0 || a.M == 1)) {
    a.by = Divisor(static_cast<uint32_t>(a.blocks));
    const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads));
    if (is_aligned(a.x, 32) && (pitch % 32 == 0 || a.M == 1))
      return launch(&quantize_kernel<T, 32>, grid, kThreads, 0, true, s, a);
    return launch(&quantize_kernel<T, 16>, grid, kThreads, 0, true, s, a);
  }
  a.by = Divisor(static_cast<uint32_t>(a.blocks / kUnits));
  const int64_t warps = static_cast<int64_t>(a.rows) * (a.blocks / kUnits);
  return launch(&quantize_by_lanes_kernel<T>,
                dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32))),
                kThreads, 0, true, s, a);
}

template <class T>
cudaError_t run_dequantize(DequantArgs a, cudaStream_t s) {
  const bool wide = is_aligned(a.q, 8) && a.ldq % 8 == 0 && a.K % 16 == 0 &&
                    rows_by(a.y, a.ldy, sizeof(T), kVecOf<T>);
  a.groups = wide ? a.K / 16 : a.K;
  a.by = Divisor(static_cast<uint32_t>(a.groups));
  const int64_t blocks = (static_cast<int64_t>(a.M) * a.groups + kThreads - 1) / kThreads;
  return launch(wide ? &dequantize_kernel<T> : &dequantize_one_kernel<T>,
                dim3(static_cast<unsigned>(blocks)), kThreads, 0, true, s, a);
}

}  // namespace
}  // namespace dlrm

extern "C" {

int64_t dlrm_fp4_scale_bytes(int64_t M, int64_t K) {
  using namespace dlrm;
  if (M < 0 || M > kMost || K < 1 || K > kMost || !fits(M, K)) return DLRM_ERR_SHAPE;
  return (M + 127) / 128 * fp4_block_tiles(K) * kFp4Tile;
}

int dlrm_quantize_fp4(const void* x, int64_t ldx, int dtype, int64_t M, int64_t K, uint8_t* q,
                      int64_t ldq, uint8_t* scale, dlrm_stream_t stream) {
  using namespace dlrm;
  if (!known_dtype(dtype)) return DLRM_ERR_ARG;
  if (M < 0 || M > kMost || K < 1 || K > kMost || ldx < K || ldq < (K + 1) / 2 || !fits(M, K))
    return DLRM_ERR_SHAPE;
  if (M == 0) return DLRM_OK;
  if (x == nullptr || q == nullptr || scale == nullptr) return DLRM_ERR_NULL;
  if (!is_aligned(x, dtype_size(dtype)) || !is_aligned(scale, 4)) return DLRM_ERR_ALIGN;
  QuantArgs a = {};
  a.x = x;
  a.q = q;
  a.scale = scale;
  a.ldx = ldx;
  a.ldq = ldq;
  a.block_tiles = fp4_block_tiles(K);
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.rows = static_cast<int>((M + 127) / 128 * 128);
  a.blocks = static_cast<int>(a.block_tiles * 4);
  const auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == DLRM_TABLE_F32 ? run_quantize<float>(a, s) : run_quantize<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

int dlrm_dequantize_fp4(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t M, int64_t K,
                        void* y, int dtype, int64_t ldy, dlrm_stream_t stream) {
  using namespace dlrm;
  if (!known_dtype(dtype)) return DLRM_ERR_ARG;
  if (M < 0 || M > kMost || K < 1 || K > kMost || ldy < K || ldq < (K + 1) / 2 || !fits(M, K))
    return DLRM_ERR_SHAPE;
  if (M == 0) return DLRM_OK;
  if (q == nullptr || scale == nullptr || y == nullptr) return DLRM_ERR_NULL;
  if (!is_aligned(y, dtype_size(dtype)) || !is_aligned(scale, 4)) return DLRM_ERR_ALIGN;
  DequantArgs a = {q, scale, y, ldq, ldy, fp4_block_tiles(K), static_cast<int>(M),
                   static_cast<int>(K), 0, Divisor()};
  const auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == DLRM_TABLE_F32 ? run_dequantize<float>(a, s) : run_dequantize<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

}  // extern "C"
