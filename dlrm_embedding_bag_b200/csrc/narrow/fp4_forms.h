// Which form of the 4-bit layer's kernels a call takes (linear_fp4.cu). Host code over sizes
// alone, so that it can be asked on the CPU.
#pragma once

#include <cstdint>

namespace dlrm {

// The forms of the tensor-core kernel, with what they take on a B200 in us besides a launch: a
// stage of a tile (`step`: 256 columns of K), a tile besides (`tile`), and what comes
// once (`once`: filling the ring, draining the last tile, joining a cluster's parts). Fitted
// to all forms at 31 shapes from 2 x 4096 x 4096 to 65536 x 592 -> 512 in a graph, weights
// from HBM; the choice was the fastest form, or within 3 % of it, at all of them.
struct Fp4Form {
  int rows_m, rows_n;  // of a tile: channels and tokens
  int units;           // of 148 SMs that walk tiles: all, or pairs
  int split;
  bool lines;          // whether it needs rows of y that start and end on 16 bytes
  double step, tile, once;
};
constexpr int kFp4Forms = 8;
constexpr Fp4Form kFp4FormOf[kFp4Forms] = {
    {128, 64, 1, 1, false, 0.349, 0.6, 0.9},
    {128, 64, 1, 2, false, 0.328, 1.9, 1.7},
    {128, 64, 1, 4, false, 0.150, 2.2, 3.0},
    {128, 128, 1, 1, false, 0.350, 1.3, 0.7},
    {128, 128, 1, 2, false, 0.331, 2.9, 1.8},
    {128, 128, 1, 4, false, 0.150, 3.2, 2.8},
    {256, 256, 2, 1, false, 0.383, 2.6, 0.8},
    {256, 256, 2, 1, true, 0.371, 1.6, 2.5},
};

// The form of least time for (M, K) rows by (N, K) weights, nkb stages of K.
// lines: rows of y start and end on 16 bytes.
inline int fp4_form(int64_t M, int64_t N, int nkb, bool lines, int sms) {
  int best = -1;
  double least = 0;
  for (int i = 0; i < kFp4Forms; ++i) {
    const Fp4Form& f = kFp4FormOf[i];
    if (f.lines && !lines) continue;
    const int64_t tiles = (M + f.rows_n - 1) / f.rows_n * ((N + f.rows_m - 1) / f.rows_m);
    // a cluster's CTAs run at the same time, and each has two K blocks at least
    if (f.split > 1 && (tiles * f.split > 128 || nkb < 2 * f.split)) continue;
    const int64_t units = sms / f.units;
    const int64_t rounds = (tiles + units - 1) / units;
    const double us = rounds * (f.step * nkb / f.split + f.tile) + f.once;
    if (best < 0 || us < least) {
      best = i;
      least = us;
    }
  }
  return best;
}

// One token and weights of up to 2^25 elements take the kernel for it (16.8 M elements 5.5 us
// and 7.0 by tensor cores, 33.5 M 10 and 10, 67 M 13.6 and 11.5).
inline bool fp4_one_token(int64_t M, int64_t N, int64_t K) {
  return M == 1 && N * K <= (int64_t{1} << 25);
}

// Its variants: channels a warp, and blocks of 32 columns that a lane has in flight. Four
// channels a warp where that leaves four warps an SM (1024 -> 8192 3.2 us, one channel 5.0; 8192 ->
// 1024 7.2 and 4.9).
struct Fp4One {
  int blocks, channels;
};
constexpr int kFp4Ones = 5;
constexpr Fp4One kFp4OneOf[kFp4Ones] = {{1, 1}, {1, 4}, {2, 1}, {2, 4}, {4, 1}};
inline int fp4_one(int64_t N, int blocks, int sms) {
  const bool many = N >= 4 * 4 * sms;
  if (blocks <= 32) return many ? 1 : 0;
  return many ? 3 : blocks <= 64 ? 2 : 4;
}

}  // namespace dlrm
