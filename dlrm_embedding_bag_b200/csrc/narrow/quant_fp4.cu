// Rows rounded to 4-bit floating point with a scale for each 32 elements, and back
// (declared in dlrm_fp4.h).
//
// Bound by reading the rows (f32: 4 bytes an element against 0.53 written). The
// scale's exponent is the largest magnitude's own, carried up where its mantissa is above
// 7/4: an integer addition to its bits. Products with powers of two are exact (where they
// do not vanish, and then the code is 0), so a code is one rounding of its element.
//
// A thread takes half a block, 16 elements, and a block's two threads exchange their
// maxima. Where rows start on 16 bytes it reads them in accesses of 16 or 32 bytes (16384 x
// 4096 bf16 28.8 us of 25.9 by their bytes; values back 28.1 of 25.9). bf16 rows that start
// anywhere it reads as the 64-bit words around them and moves those down (60000 x 1001 37.6 us of
// 23.2, the integer pipe that moves them at 76 %; by neighbouring elements through shared memory
// 43.8). f32 rows that start anywhere lanes
// read by neighbouring elements, whole lines, and lay them out in shared memory from
// where each takes its own 16 (45.3 us of 41.5); values go back the same way, or in
// aligned words of the row (below).
#include <algorithm>
#include <climits>

#include "fp4_common.cuh"
#include "sectors.cuh"
#include "tokens/common.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr uint32_t kInfBits = 0x7f800000u;

struct QuantArgs {
  const void* x;
  const void* end;  // behind the last row's last element
  uint8_t* q;
  uint8_t* scale;
  int64_t ldx, ldq, block_tiles;
  int M, K;
  int rows;    // with the scales' padding: a multiple of 128
  int blocks;  // of a row
  Divisor by;  // what a row is cut into: blocks, or pieces
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

// Eight elements as codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t codes_of(const Pair (&x)[4]) {
  const float2 a = parts(x[0]), b = parts(x[1]), c = parts(x[2]), d = parts(x[3]);
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// The larger magnitudes of two pairs of bf16, NaN if one is; the signs say nothing.
__device__ __forceinline__ uint32_t max_abs_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 elements from p, of which `left` are the row's, as words; what is not reads as zero.
// BYTES: 16 or 32 at a time.
template <class T, int BYTES>
__device__ __forceinline__ void load_half_block(const T* p, int left, uint32_t (&w)[4 * sizeof(T)]) {
  constexpr int kPieces = sizeof(T);      // of 16 bytes
  constexpr int kOfPiece = 16 / sizeof(T);  // elements
  if (BYTES == 32 && left >= 16) {
#pragma unroll
    for (int i = 0; i < kPieces; i += 2)
      load_32_bytes(p + i * kOfPiece, *reinterpret_cast<uint32_t(*)[8]>(w + 4 * i));
    return;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const T* at = p + i * kOfPiece;
    const int in = left - i * kOfPiece;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in >= kOfPiece) {
      v = *reinterpret_cast<const uint4*>(at);
    } else if (in > 0) {
      uint32_t e[4] = {};
#pragma unroll
      for (int k = 0; k < kOfPiece; ++k)
        if (k < in) {
          if constexpr (sizeof(T) == 4)
            e[k] = __float_as_uint(at[k]);
          else
            e[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(at)[k]) << (16 * (k % 2));
        }
      v = make_uint4(e[0], e[1], e[2], e[3]);
    }
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
}

// The same of bf16 rows that start anywhere: the five 64-bit words of the matrix around the 16
// elements (some of them its neighbours' too, from L1), moved down by their start. Where
// those reach past the matrix, and only there, element by element.
__device__ __forceinline__ void load_half_block_anywhere(const QuantArgs& a, const __nv_bfloat16* p,
                                                         int left, uint32_t (&w)[8]) {
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 7;  // even
  const uint2* words = reinterpret_cast<const uint2*>(reinterpret_cast<uintptr_t>(p) - off);
  if (words >= a.x && words + 5 <= a.end) {
    uint32_t v[10];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint2 r = words[i];
      v[2 * i] = r.x, v[2 * i + 1] = r.y;
    }
#pragma unroll
    for (int k = 0; k < 9; ++k) v[k] = off & 4 ? v[k + 1] : v[k];
    const uint32_t which = off & 2 ? 0x5432 : 0x3210;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __byte_perm(v[k], v[k + 1], which);
    if (left < 16) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        w[k] &= (2 * k < left ? 0xffffu : 0u) | (2 * k + 1 < left ? 0xffff0000u : 0u);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (k < left)
      w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[k]) << (16 * (k % 2));
}

// A thread's half block: its words rounded, codes and (a block's first thread) the scale
// written. Every lane of a warp comes here; in: whether the row has such a block, or a
// scale tile has it beside the row's.
template <class T>
__device__ __forceinline__ void round_half_block(const QuantArgs& a, int row, int block, int half,
                                                 bool in, const uint32_t (&w)[4 * sizeof(T)]) {
  constexpr int kWords = 4 * sizeof(T);
  const int c = block * 32 + half * 16;
  uint32_t top;
  if constexpr (sizeof(T) == 4) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kWords; k += 2)
      t = max_abs(t, __uint_as_float(w[k]), __uint_as_float(w[k + 1]));
    top = __float_as_uint(t);
  } else {
    uint32_t two = w[0];
#pragma unroll
    for (int k = 1; k < kWords; ++k) two = max_abs_bf16(two, w[k]);
    two &= 0x7fff7fffu;
    top = max(two & 0xffff0000u, two << 16);
  }
  top = max(top, __shfl_xor_sync(kFull, top, 1));
  if (!in) return;
  const uint32_t byte = scale_byte(top);
  if (half == 0) a.scale[fp4_scale_at(a.block_tiles, row, block)] = static_cast<uint8_t>(byte);
  if (row >= a.M || c >= a.K) return;
  const Pair inv = both(inverse_of(byte));
  uint32_t out[2] = {};
  if (byte != 255u) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Pair x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4)
          x[k] = pair(__uint_as_float(w[8 * h + 2 * k]), __uint_as_float(w[8 * h + 2 * k + 1]));
        else
          x[k] = pair(__uint_as_float(w[4 * h + k] << 16), __uint_as_float(w[4 * h + k] & 0xffff0000u));
        x[k] = mul(x[k], inv);
      }
      out[h] = codes_of(x);
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

// BYTES: of an access that rows allow; 2: bf16 rows that start anywhere.
template <class T, int BYTES>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t two = i >> 1;
  const int row = static_cast<int>(a.by.of(two));
  const int block = static_cast<int>(two - static_cast<int64_t>(row) * a.blocks);
  const int half = static_cast<int>(i & 1);
  const int c = block * 32 + half * 16;
  uint32_t w[4 * sizeof(T)] = {};
  if (row < a.M && c < a.K) {
    const T* p = static_cast<const T*>(a.x) + row * a.ldx + c;
    if constexpr (BYTES == 2)
      load_half_block_anywhere(a, p, a.K - c, w);
    else
      load_half_block<T, BYTES>(p, a.K - c, w);
  }
  round_half_block<T>(a, row, block, half, row < a.rows, w);
  // the last block's thread ends the scale tile's four
  if (half == 0 && row < a.rows && block == a.blocks - 1)
    for (int k = block + 1; k & 3; ++k) a.scale[fp4_scale_at(a.block_tiles, row, k)] = 0;
}

// Where a group of lanes lays a piece of a row out, 16 elements of each lane with 16 bytes
// between them and the next lane's: 128-bit accesses of neighbouring lanes then meet in no
// bank (80 or 48 bytes apart).
template <class T>
struct Staged {
  static constexpr int kLane = 16 + 16 / sizeof(T);  // elements
  T v[32 * kLane];
  static __device__ __forceinline__ int at(int e) { return e / 16 * kLane + e % 16; }
};

// G lanes take 16 G columns of a row.
template <class T, int G>
__global__ void __launch_bounds__(kThreads) quantize_staged_kernel(const QuantArgs a, int pieces) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  static_assert(G % 8 == 0, "whole scale tiles");
  __shared__ alignas(16) Staged<T> staged[kThreads / 32];
  const int lane = threadIdx.x & 31, in = lane % G;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / G;
  const int row = static_cast<int>(a.by.of(unit));
  const int piece = static_cast<int>(unit - static_cast<int64_t>(row) * pieces);
  const int c0 = piece * 16 * G;
  const int left = row < a.M ? a.K - c0 : 0;  // columns of the piece
  const T* x = static_cast<const T*>(a.x) + row * a.ldx + c0 + in;
  T v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = j * G + in < left ? x[j * G] : T(0.f);
  T* mine = staged[threadIdx.x >> 5].v + lane / G * (G * Staged<T>::kLane);
#pragma unroll
  for (int j = 0; j < 16; ++j) mine[Staged<T>::at(j * G + in)] = v[j];
  __syncwarp();
  uint32_t w[4 * sizeof(T)];
  const uint4* own = reinterpret_cast<const uint4*>(mine + Staged<T>::at(16 * in));
#pragma unroll
  for (int k = 0; k < static_cast<int>(sizeof(T)); ++k) {
    const uint4 r = own[k];
    w[4 * k] = r.x, w[4 * k + 1] = r.y, w[4 * k + 2] = r.z, w[4 * k + 3] = r.w;
  }
  const int block = piece * (G / 2) + in / 2;
  round_half_block<T>(a, row, block, in & 1, row < a.rows && block < 4 * a.block_tiles, w);
}

// Back to values.
struct DequantArgs {
  const uint8_t* q;
  const uint8_t* scale;
  void* y;
  int64_t ldq, ldy, block_tiles;
  int M, K;
  int groups;  // what a row is cut into: half blocks, or pieces
  Divisor by;  // groups
};

// What a scale byte stands for, as the bits of f32 (its upper half those of bf16).
__device__ __forceinline__ uint32_t scale_bits(uint32_t byte) {
  return byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23;
}

// Sixteen codes (two words) as pairs of bf16 numbers without their scales: four at a time
// are looked up, whose upper and lower bytes are one byte permutation each.
__device__ __forceinline__ void pairs_of(const uint32_t (&codes)[2], uint32_t (&two)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = codes[i / 2] >> (16 * (i % 2));
    const uint32_t at = c & 0x7777u;
    uint32_t signs;  // bytes of 0x80, or 0xff where a code's sign bit is set
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(signs) : "r"(0x80808080u), "r"(c));
    // 0, 0.5, 1, 1.5 and 2, 3, 4, 6
    const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, at) | (signs << 1 & 0x80808080u);
    const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, at);
    two[2 * i] = __byte_perm(lo, hi, 0x5140), two[2 * i + 1] = __byte_perm(lo, hi, 0x7362);
  }
}
// Products of two bf16 numbers and powers of two: as exact as in f32.
__device__ __forceinline__ uint32_t scaled(uint32_t two, uint32_t scales) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(two), "r"(scales));
  return r;
}

// Sixteen codes times their scale as T, rounded once, eight words of bf16 or sixteen of f32.
template <class T>
__device__ __forceinline__ void values_of(const uint32_t (&codes)[2], uint32_t byte,
                                          uint32_t (&v)[4 * sizeof(T)]) {
  const uint32_t scale = scale_bits(byte);
  uint32_t two[8];
  pairs_of(codes, two);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[i] = scaled(two[i], scale >> 16 | scale);
    } else {
      const float2 f = parts(mul(pair(__uint_as_float(two[i] << 16), __uint_as_float(two[i] & 0xffff0000u)),
                                 both(__uint_as_float(scale))));
      v[2 * i] = __float_as_uint(f.x), v[2 * i + 1] = __float_as_uint(f.y);
    }
  }
}

template <class T, bool SECTORS>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = a.by.of(i);
  if (row >= a.M) return;
  const int c = static_cast<int>(i - row * a.groups) * 16;
  const uint32_t byte = a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), c / 32)];
  const uint2 r = *reinterpret_cast<const uint2*>(a.q + row * a.ldq + c / 2);
  const uint32_t codes[2] = {r.x, r.y};
  uint32_t v[4 * sizeof(T)];
  values_of<T>(codes, byte, v);
  T* y = static_cast<T*>(a.y) + row * a.ldy + c;
  if constexpr (SECTORS) {
    store_sector_words(y, v);
  } else {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      reinterpret_cast<uint4*>(y)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// Eight bytes of a row's codes from byte `at` on (a multiple of 8, negative in front of the
// row). WHOLE: rows start on 8 bytes; what lies between a row's codes and the next one may
// come with them.
template <bool WHOLE>
__device__ __forceinline__ uint2 load_16_codes(const DequantArgs& a, int64_t row, int at) {
  const int bytes = (a.K + 1) / 2;
  if (at < 0 || at >= bytes) return make_uint2(0, 0);
  const uint8_t* q = a.q + row * a.ldq + at;
  if (WHOLE && (at + 8 <= bytes || row < a.M - 1)) return *reinterpret_cast<const uint2*>(q);
  uint32_t w[2] = {};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (at + k < bytes) w[k / 4] |= static_cast<uint32_t>(q[k]) << (8 * (k % 4));
  return make_uint2(w[0], w[1]);
}

// bf16 rows that start anywhere: a thread takes the row's part of 32 aligned bytes of y, 16
// columns that may begin inside a half block and lie in two blocks.
template <bool WHOLE>
__global__ void __launch_bounds__(kThreads) dequantize_anywhere_kernel(const DequantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = a.by.of(i);
  if (row >= a.M) return;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + row * a.ldy;
  const int before = static_cast<int>(reinterpret_cast<uintptr_t>(y) & 31) / 2;
  const int c = static_cast<int>(i - row * a.groups) * 16 - before;
  if (c >= a.K) return;
  const int c16 = c & ~15;
  const uint2 lo = load_16_codes<WHOLE>(a, row, c16 / 2);
  const uint2 hi = load_16_codes<WHOLE>(a, row, c16 / 2 + 8);
  const int block = c >> 5, cut = 32 - (c & 31);  // columns of the first block
  const uint32_t b0 = block >= 0 ? a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), block)] : 0u;
  const uint32_t b1 = cut < 16 && c + cut < a.K
                          ? a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), block + 1)]
                          : 0u;
  const bool upper = c & 8;
  const uint32_t x0 = upper ? lo.y : lo.x, x1 = upper ? hi.x : lo.y, x2 = upper ? hi.y : hi.x;
  const uint32_t codes[2] = {__funnelshift_r(x0, x1, 4 * (c & 7)),
                             __funnelshift_r(x1, x2, 4 * (c & 7))};
  uint32_t v[8];
  pairs_of(codes, v);
  const uint32_t s0 = scale_bits(b0), s1 = scale_bits(b1);
  const uint32_t of_first = s0 >> 16 | s0, of_both = s0 >> 16 | s1, of_second = s1 >> 16 | s1;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    v[k] = scaled(v[k], 2 * k + 1 < cut ? of_first : 2 * k < cut ? of_both : of_second);
  if (c >= 0 && c + 16 <= a.K) {
    store_sector_words(y + c, v);
    return;
  }
  // a row's ends: pairs, and the one element that is left over of each
  const int first = max(-c, 0), last = min(a.K - c, 16);
  uint32_t* at = reinterpret_cast<uint32_t*>(y + c);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (2 * k >= first && 2 * k + 2 <= last) at[k] = v[k];
  uint16_t* one = reinterpret_cast<uint16_t*>(at);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (first == 2 * k + 1) one[2 * k + 1] = static_cast<uint16_t>(v[k] >> 16);
    if (last == 2 * k + 1) one[2 * k] = static_cast<uint16_t>(v[k]);
  }
}

// G lanes take 16 G columns of a row, from one in front of it on where a bf16 row starts
// between two words, so that all but its ends are stored as words (60000 x 1001
// 40.1 us, by elements 41.4; 30000 x 1000 18.8 and 21.3; the integer pipe at 78 %).
template <class T, int G>
__global__ void __launch_bounds__(kThreads) dequantize_staged_kernel(const DequantArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kWords = 4 * sizeof(T), kOfWord = 4 / sizeof(T);
  __shared__ alignas(16) Staged<T> staged[kThreads / 32];
  const int lane = threadIdx.x & 31, in = lane % G;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / G;
  const int64_t row = a.by.of(unit);
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const int before = sizeof(T) == 2 ? static_cast<int>(reinterpret_cast<uintptr_t>(y) >> 1 & 1) : 0;
  const int c0 = static_cast<int>(unit - row * a.groups) * 16 * G - before;
  const int c = c0 + before + 16 * in;  // the lane's half block
  const int left = row < a.M ? a.K - c0 : 0;
  uint32_t w[2] = {}, byte = 0;
  const uint8_t* q = a.q + row * a.ldq + c / 2;
  if (row < a.M && c < a.K) {
    byte = a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), c / 32)];
    const int bytes = (a.K - c + 1) / 2;
    if (bytes >= 8 && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
      const uint2 r = *reinterpret_cast<const uint2*>(q);
      w[0] = r.x, w[1] = r.y;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < bytes) w[k / 4] |= static_cast<uint32_t>(q[k]) << (8 * (k % 4));
    }
  }
  uint32_t v[kWords];
  if (sizeof(T) == 2 && before != 0) {
    // the column in front of the half block, and all of that but its last one
    uint32_t code = 0, other = 0;
    if (row < a.M && c > 0 && c <= a.K) {
      code = q[-1] >> 4;
      other = a.scale[fp4_scale_at(a.block_tiles, static_cast<int>(row), (c - 1) / 32)];
    }
    const uint32_t moved[2] = {w[0] << 4 | code, __funnelshift_l(w[0], w[1], 4)};
    uint32_t two[8];
    pairs_of(moved, two);
    const uint32_t scale = scale_bits(byte);
    v[0] = scaled(two[0], scale_bits(other) >> 16 | scale);
#pragma unroll
    for (int k = 1; k < 8; ++k) v[k] = scaled(two[k], scale >> 16 | scale);
  } else {
    values_of<T>(w, byte, v);
  }
  T* mine = staged[threadIdx.x >> 5].v + lane / G * (G * Staged<T>::kLane);
  uint4* own = reinterpret_cast<uint4*>(mine + Staged<T>::at(16 * in));
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
    own[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const int e = (j * G + in) * kOfWord;
    if (c0 + e >= 0 && e + kOfWord <= left)
      *reinterpret_cast<uint32_t*>(y + c0 + e) =
          *reinterpret_cast<const uint32_t*>(mine + Staged<T>::at(e));
  }
  if (sizeof(T) == 2 && in == 0) {
    if (c0 < 0 && left > 0) y[0] = mine[Staged<T>::at(1)];
    if (left > 0 && left <= 16 * G && left % 2 != 0) y[a.K - 1] = mine[Staged<T>::at(left - 1)];
  }
}

constexpr int64_t kMost = INT_MAX - 1024;
// Largest M * K (rounded up to whole scale tiles): no grid leaves 2^31 blocks and no
// quotient its Divisor's range. (180 GB hold 2^37 elements of bf16.)
constexpr int64_t kMostElements = int64_t{1} << 38;

bool fits(int64_t M, int64_t K) {
  return (M + 127) / 128 * fp4_block_tiles(K) <= kMostElements / (128 * 128) && M * K < kMostElements;
}

unsigned grid_of(int64_t things, int64_t a_block) {
  return static_cast<unsigned>((things + a_block - 1) / a_block);
}

template <class T, int G>
cudaError_t run_staged(QuantArgs a, cudaStream_t s) {
  const int pieces = (a.blocks + G / 2 - 1) / (G / 2);
  a.by = Divisor(static_cast<uint32_t>(pieces));
  return launch(&quantize_staged_kernel<T, G>,
                dim3(grid_of(static_cast<int64_t>(a.rows) * pieces * G, kThreads)), kThreads, 0,
                true, s, a, pieces);
}
template <class T, int G>
cudaError_t run_staged(DequantArgs a, cudaStream_t s) {
  // bf16 rows may begin between two words
  const bool words = sizeof(T) == 4 || (is_aligned(a.y, 4) && (a.ldy % 2 == 0 || a.M == 1));
  a.groups = (a.K + (words ? 0 : 1) + 16 * G - 1) / (16 * G);
  a.by = Divisor(static_cast<uint32_t>(a.groups));
  return launch(&dequantize_staged_kernel<T, G>,
                dim3(grid_of(static_cast<int64_t>(a.M) * a.groups * G, kThreads)), kThreads, 0,
                true, s, a);
}
// The lanes of a piece: as few as cover a short row, and no more columns past a long one's end than
// a quarter warp's.
int lanes_of_piece(int K) {
  const int tail = (K - 1) % 512 + 1;
  if (K <= 128 || (K < 2048 && tail <= 128)) return 8;
  return K <= 256 || (K < 4096 && tail <= 256) ? 16 : 32;
}
template <class T, class Args>
cudaError_t run_staged_by(const Args& a, cudaStream_t s) {
  const int lanes = lanes_of_piece(a.K);
  if (lanes == 8) return run_staged<T, 8>(a, s);
  return lanes == 16 ? run_staged<T, 16>(a, s) : run_staged<T, 32>(a, s);
}

template <class T>
cudaError_t run_quantize(QuantArgs a, cudaStream_t s) {
  const int64_t pitch = a.ldx * static_cast<int64_t>(sizeof(T));
  const bool wide = is_aligned(a.x, 16) && (pitch % 16 == 0 || a.M == 1);
  if constexpr (sizeof(T) == 4) {
    if (!wide) return run_staged_by<T>(a, s);
  }
  a.by = Divisor(static_cast<uint32_t>(a.blocks));
  const dim3 grid(grid_of(static_cast<int64_t>(a.rows) * a.blocks * 2, kThreads));
  if constexpr (sizeof(T) == 2) {
    if (!wide) return launch(&quantize_kernel<T, 2>, grid, kThreads, 0, true, s, a);
  }
  const bool wider = is_aligned(a.x, 32) && (pitch % 32 == 0 || a.M == 1);
  return launch(wider ? &quantize_kernel<T, 32> : &quantize_kernel<T, 16>, grid, kThreads, 0, true,
                s, a);
}

template <class T>
cudaError_t run_dequantize(DequantArgs a, cudaStream_t s) {
  const bool wide = is_aligned(a.q, 8) && a.ldq % 8 == 0 && a.K % 16 == 0 &&
                    rows_by(a.y, a.ldy, sizeof(T), kVecOf<T>);
  if constexpr (sizeof(T) == 2) {
    // Where the pieces have half as many columns again as the row, a thread for each 32 bytes of
    // y: 20 M elements by 63 columns 21.8 us (by pieces of 128: 31.7), by 257 18.1 (512: 26.8), by
    // 13 41.5 (128: 145); but by 200 19.1 (256: 17.1) and by 1001 17.3 (1024: 14.1), for a
    // row's ends are single stores.
    const int64_t piece = 16 * lanes_of_piece(a.K);
    if (!wide && (a.K + piece - 1) / piece * piece * 2 > int64_t{3} * a.K) {
      a.groups = (a.K + 30) / 16;
      a.by = Divisor(static_cast<uint32_t>(a.groups));
      const bool whole = is_aligned(a.q, 8) && a.ldq % 8 == 0;
      return launch(whole ? &dequantize_anywhere_kernel<true> : &dequantize_anywhere_kernel<false>,
                    dim3(grid_of(static_cast<int64_t>(a.M) * a.groups, kThreads)), kThreads, 0, true,
                    s, a);
    }
  }
  if (!wide) return run_staged_by<T>(a, s);
  a.groups = a.K / 16;
  a.by = Divisor(static_cast<uint32_t>(a.groups));
  const int64_t units = static_cast<int64_t>(a.M) * a.groups;
  const bool sectors = is_aligned(a.y, 32) && a.ldy * sizeof(T) % 32 == 0;
  return launch(sectors ? &dequantize_kernel<T, true> : &dequantize_kernel<T, false>,
                dim3(grid_of(units, kThreads)), kThreads, 0, true, s, a);
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
  a.end = static_cast<const uint8_t*>(x) + ((M - 1) * ldx + K) * dtype_size(dtype);
  a.q = q;
  a.scale = scale;
  a.ldx = ldx;
  a.ldq = ldq;
  a.block_tiles = fp4_block_tiles(K);
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.rows = static_cast<int>((M + 127) / 128 * 128);
  a.blocks = static_cast<int>((K + 31) / 32);
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
