// What the kernels of the 4-bit matrices share (the format is in dlrm_fp4.h).
#pragma once

#include <cstdint>

#include "dlrm_fp4.h"

namespace dlrm {

constexpr int kFp4Tile = 512;  // bytes of a scale tile: 128 rows x 4 blocks

// Block tiles of a row, and where the scale of (row, block) lies.
__host__ __device__ inline int64_t fp4_block_tiles(int64_t K) { return (K + 127) / 128; }
__host__ __device__ inline int64_t fp4_scale_at(int64_t block_tiles, int row, int block) {
  return ((row >> 7) * block_tiles + (block >> 2)) * kFp4Tile + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (block & 3);
}

// n / d by a product, for n * d < 2^64: with m = floor(2^64 / d) + 1, n m / 2^64 is
// above n / d by less than 1 / d.
struct Divisor {
  uint64_t m = 0;  // 0: d is 1
  Divisor() = default;
  explicit Divisor(uint32_t d) : m(d == 1 ? 0 : ~uint64_t{0} / d + 1) {}
  __device__ __forceinline__ int64_t of(int64_t n) const {
    return m == 0 ? n : static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(n), m));
  }
};

}  // namespace dlrm
