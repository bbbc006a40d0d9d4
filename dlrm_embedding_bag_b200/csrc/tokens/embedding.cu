// Embedding rows by token id, and the table's gradient by sorted tokens
// (declared in dlrm_tokens.h).
#include <algorithm>
#include <climits>

#include "common.h"
#include "dlrm_tokens.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Lookup: Y[t] = scale * W[ids[t]].
//
// G lanes walk one row, VEC elements each per step; a group takes kRowsInFlight
// tokens at a time, so that as many row loads are in the air before the first
// is used. No arithmetic to speak of: bound by the bytes of the rows read and
// written.

constexpr int kLookupThreads = 256;
constexpr int kRowsInFlight = 4;

struct LookupArgs {
  const void* table;
  int64_t ldw;
  const int32_t* ids;
  void* out;
  int64_t ldo;
  int rows, D, T, pad;
  float scale;
  int32_t* status;
};

template <class In, class Out, int VEC, int G>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const LookupArgs a) {
  const In* W = static_cast<const In*>(a.table);
  Out* Y = static_cast<Out*>(a.out);
  const int q = threadIdx.x % G;
  const int64_t group = (static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x) / G;
  const int64_t t0 = group * kRowsInFlight;
  int id[kRowsInFlight];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    id[u] = -1;  // nothing to write
    if (t0 + u < a.T) {
      const int r = __ldg(a.ids + t0 + u);
      const bool in = static_cast<unsigned>(r) < static_cast<unsigned>(a.rows);
      if (!in && a.status != nullptr && q == 0) atomicOr(a.status, DLRM_FLAG_INDEX_OOB);
      id[u] = (in && r != a.pad) ? r : a.rows;  // `rows`: a row of zeros
    }
  }
  for (int c = q * VEC; c < a.D; c += G * VEC) {
    float v[kRowsInFlight][VEC];
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[u][e] = 0.f;
      if (id[u] >= 0 && id[u] < a.rows) {
        load_f32<In, VEC>(W + static_cast<int64_t>(id[u]) * a.ldw + c, v[u]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[u][e] *= a.scale;
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsInFlight; ++u)
      if (id[u] >= 0) store_f32<Out, VEC>(Y + (t0 + u) * a.ldo + c, v[u]);
  }
}

template <class In, class Out, int VEC, int G>
cudaError_t run_lookup(const LookupArgs& a, cudaStream_t stream) {
  constexpr int per_block = kLookupThreads / G * kRowsInFlight;
  const int64_t blocks = (static_cast<int64_t>(a.T) + per_block - 1) / per_block;
  lookup_kernel<In, Out, VEC, G><<<static_cast<unsigned>(blocks), kLookupThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <class In, class Out>
cudaError_t run_lookup_shape(const LookupArgs& a, bool vec, cudaStream_t stream) {
  constexpr int V = kVecOf<In>;
  if (!vec) return run_lookup<In, Out, 1, 32>(a, stream);
  const int chunks = a.D / V;
  if (chunks <= 4) return run_lookup<In, Out, V, 4>(a, stream);
  if (chunks <= 8) return run_lookup<In, Out, V, 8>(a, stream);
  if (chunks <= 16) return run_lookup<In, Out, V, 16>(a, stream);
  return run_lookup<In, Out, V, 32>(a, stream);
}

// ---------------------------------------------------------------------------
// Gradient, step 1: the tokens sorted by id, stable.
//
// Least-significant-digit radix sort of (key, token) pairs with digits of at
// most 8 bits over the bits that `rows` needs. A pass is two kernels: every
// block counts the digits of its stretch of pairs, then every block adds up
// the counts of all digits and of the blocks before it, and moves its pairs.
// Padding and out-of-range ids take the key `rows` and so come last.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kRadix = 256;
constexpr int kSortMaxBlocks = 148;

struct SortArgs {
  const int32_t* ids;  // first pass: the tokens' ids; later passes read `in`
  const uint2* in;     // (key, token)
  uint2* out;
  uint32_t* counts;  // [block][kRadix]
  int T, rows, pad;
  int shift, bits;
  int per;  // pairs of a block, a multiple of kSortThreads
  int32_t* status;
};

__device__ __forceinline__ uint2 sort_pair(const SortArgs& a, int i) {
  if (a.ids == nullptr) return a.in[i];
  const int r = __ldg(a.ids + i);
  const bool in = static_cast<unsigned>(r) < static_cast<unsigned>(a.rows);
  const uint32_t key = (in && r != a.pad) ? r : a.rows;
  return make_uint2(key, static_cast<uint32_t>(i));
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a) {
  __shared__ uint32_t cnt[kRadix];
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < kRadix) cnt[tid] = 0;
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.per;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int64_t i0 = begin; i0 < begin + a.per; i0 += kSortThreads) {
    const int64_t i = i0 + tid;
    const bool live = i < a.T;
    uint32_t digit = kRadix;  // of no pair
    if (live) {
      if (a.ids != nullptr && a.status != nullptr &&
          static_cast<unsigned>(__ldg(a.ids + i)) >= static_cast<unsigned>(a.rows))
        atomicOr(a.status, DLRM_FLAG_INDEX_OOB);
      digit = (sort_pair(a, static_cast<int>(i)).x >> a.shift) & mask;
    }
    const unsigned peers = __match_any_sync(kFull, digit);
    if (live && lane == __ffs(peers) - 1) atomicAdd(&cnt[digit], __popc(peers));
  }
  __syncthreads();
  if (tid < kRadix) a.counts[static_cast<int64_t>(blockIdx.x) * kRadix + tid] = cnt[tid];
}

__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const SortArgs a) {
  __shared__ uint32_t at[kSortWarps][kRadix];  // a warp's next place for each digit
  __shared__ uint32_t total[kSortThreads / kRadix][kRadix], before[kSortThreads / kRadix][kRadix];
  __shared__ uint32_t warp_sum[kRadix / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t mask = (1u << a.bits) - 1;
  for (int d = lane; d < kRadix; d += 32) at[warp][d] = 0;
  __syncwarp();
  // every warp counts the digits of its own stretch of pairs
  const int per_warp = a.per / kSortWarps;
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.per + warp * per_warp;
  for (int j = 0; j < per_warp; j += 32) {
    const int64_t i = begin + j + lane;
    const bool live = i < a.T;
    const uint32_t digit = live ? (sort_pair(a, static_cast<int>(i)).x >> a.shift) & mask : kRadix;
    const unsigned peers = __match_any_sync(kFull, digit);
    if (live && lane == __ffs(peers) - 1) at[warp][digit] += __popc(peers);
    __syncwarp();
  }
  // digit d: pairs in all blocks, and in the blocks before this one
  const int d = tid % kRadix, part = tid / kRadix;
  uint32_t all = 0, mine = 0;
  for (int b = part; b < static_cast<int>(gridDim.x); b += kSortThreads / kRadix) {
    const uint32_t n = a.counts[static_cast<int64_t>(b) * kRadix + d];
    all += n;
    mine += b < static_cast<int>(blockIdx.x) ? n : 0;
  }
  total[part][d] = all;
  before[part][d] = mine;
  __syncthreads();
  uint32_t place = 0, scan = 0;
  if (tid < kRadix) {
    all = 0;
    for (int p = 0; p < kSortThreads / kRadix; ++p) {
      all += total[p][d];
      place += before[p][d];
    }
    scan = all;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(kFull, scan, o);
      if (lane >= o) scan += n;
    }
    if (lane == 31) warp_sum[warp] = scan;
  }
  __syncthreads();
  if (tid < kRadix) {
    for (int w = 0; w < warp; ++w) scan += warp_sum[w];
    place += scan - all;
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t n = at[w][d];
      at[w][d] = place;
      place += n;
    }
  }
  __syncthreads();
  for (int j = 0; j < per_warp; j += 32) {
    const int64_t i = begin + j + lane;
    const bool live = i < a.T;
    uint2 pair = make_uint2(0, 0);
    uint32_t digit = kRadix;
    if (live) {
      pair = sort_pair(a, static_cast<int>(i));
      digit = (pair.x >> a.shift) & mask;
    }
    const unsigned peers = __match_any_sync(kFull, digit);
    if (live) {
      const uint32_t to = at[warp][digit] + __popc(peers & ((1u << lane) - 1));
      a.out[to] = pair;
    }
    __syncwarp();
    if (live && lane == __ffs(peers) - 1) at[warp][digit] += __popc(peers);
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// Gradient, step 2: sums over runs of equal ids.
//
// The sorted tokens are cut into chunks; a group of G lanes sums a chunk's rows
// (a window of G * VEC columns of them) run by run in sorted order, eight rows
// in flight. A run that lies inside its chunk is written at once. One that
// crosses a border leaves parts, which meet in two levels: the groups of a
// block, whose chunks follow each other, in shared memory; then blocks through
// one f32 row each for a run that came in from the left (slot 0) and one that
// goes out to the right (slot 1), added up by the join kernel. The order of
// every sum is fixed by the sizes.

constexpr int kSumThreads = 256;
constexpr int kSumInFlight = 8;
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 128;  // columns of a join block: four a lane

struct SumArgs {
  const void* grad;
  int64_t ldg;
  const uint2* sorted;
  float* part;  // [block of chunks][2][Dp]
  int64_t Dp;
  void* out;
  int64_t ldo;
  int T, L, rows, D;
  int chunk;      // tokens of a group, a multiple of kSumInFlight
  int per_block;  // tokens of a block
  int nblocks;    // of a window
  int windows;
  float scale;
  int out_bf16, accumulate;
};

template <int VEC>
__device__ __forceinline__ void put_row(const SumArgs& a, uint32_t row, int c,
                                        const float (&sum)[VEC]) {
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = sum[e] * a.scale;
  const int64_t at = static_cast<int64_t>(row) * a.ldo + c;
  if (a.out_bf16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.out) + at;
    if (a.accumulate) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] += static_cast<float>(p[e]);
    }
    store_f32<__nv_bfloat16, VEC>(p, v);
  } else {
    float* p = static_cast<float*>(a.out) + at;
    if (a.accumulate) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] += p[e];
    }
    store_f32<float, VEC>(p, v);
  }
}

template <class In, int VEC, int G>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumArgs a) {
  constexpr int NG = kSumThreads / G;  // groups, with chunks that follow each other
  constexpr int U = G < kSumInFlight ? G : kSumInFlight;
  __shared__ float head[NG][G * VEC], tail[NG][G * VEC];
  __shared__ uint32_t first[NG], last[NG];
  const int q = threadIdx.x % G, g = threadIdx.x / G, base = (threadIdx.x & 31) / G * G;
  const int block = blockIdx.x / a.windows;
  const int c = (static_cast<int>(blockIdx.x % a.windows) * G + q) * VEC;
  const bool cols = c < a.D;
  const int64_t begin = static_cast<int64_t>(block) * a.per_block + static_cast<int64_t>(g) * a.chunk;
  const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(a.chunk), a.T - begin)));
  const In* grad = static_cast<const In*>(a.grad);
  const uint32_t none = a.rows;
  const uint32_t left = (n > 0 && begin > 0) ? a.sorted[begin - 1].x : none;
  const uint32_t right = (n > 0 && begin + n < a.T) ? a.sorted[begin + n].x : none;
  if (q == 0) {
    first[g] = n > 0 ? a.sorted[begin].x : none;
    last[g] = n > 0 ? a.sorted[begin + n - 1].x : none;
  }
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  uint32_t cur = none;  // key of the run being summed; none before the first
  bool inside = false;  // it began in this chunk
  // every lane of the warp takes the same number of steps: shuffles span it
  for (int j0 = 0; j0 < a.chunk; j0 += G) {
    uint32_t key = none, row = 0;
    if (j0 + q < n) {
      const uint2 p = a.sorted[begin + j0 + q];
      key = p.x;
      row = p.y / static_cast<uint32_t>(a.L);
    }
    const int steps = min(G, a.chunk - j0);
    for (int u0 = 0; u0 < steps; u0 += U) {
      float v[U][VEC];
      uint32_t k[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        k[u] = __shfl_sync(kFull, key, base + u0 + u);
        const uint32_t r = __shfl_sync(kFull, row, base + u0 + u);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[u][e] = 0.f;
        if (k[u] != none && cols)
          load_f32<In, VEC>(grad + static_cast<int64_t>(r) * a.ldg + c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k[u] != cur) {
          // the run before this token ends here
          if (cur != none) {
            if (!inside)
              store_f32<float, VEC>(&head[g][q * VEC], acc);
            else if (cols)
              put_row<VEC>(a, cur, c, acc);
          }
          inside = k[u] != left || j0 + u0 + u > 0;
          cur = k[u];
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += v[u][e];
      }
    }
  }
  const bool out_right = cur != none && cur == right;  // the last run goes on
  if (cur != none) {
    if (!inside)
      store_f32<float, VEC>(&head[g][q * VEC], acc);
    else if (out_right)
      store_f32<float, VEC>(&tail[g][q * VEC], acc);
    else if (cols)
      put_row<VEC>(a, cur, c, acc);
  }
  // the last group's lanes alone know whether the block's last run goes on
  const bool block_goes_on = __syncthreads_or(g == NG - 1 && out_right);
  auto goes_on = [&](int j) {  // group j's last run does not end with it
    return j + 1 < NG ? last[j] != none && last[j] == first[j + 1] : block_goes_on;
  };
  auto one_run = [&](int j) { return first[j] == last[j] && goes_on(j); };
  float* part = a.part + static_cast<int64_t>(block) * 2 * a.Dp + c;
  if (inside && out_right) {
    // a run that begins in this group: its parts to the right
    bool open = true;
    int j = g + 1;
    for (; j < NG && open; ++j) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += head[j][q * VEC + e];
      open = one_run(j);
    }
    if (cols) {
      if (open)
        store_f32<float, VEC>(part + a.Dp, acc);
      else
        put_row<VEC>(a, cur, c, acc);
    }
  }
  if (g == 0 && n > 0 && first[0] != none && first[0] == left) {
    // the run that came in from the block before
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = head[0][q * VEC + e];
    for (int j = 0; j + 1 < NG && one_run(j); ++j) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += head[j + 1][q * VEC + e];
    }
    if (cols) store_f32<float, VEC>(part, acc);
  }
}

// The runs that begin in a block of chunks and go on past its end: their parts,
// added by the warps of a block in turn, for a window of columns.
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const SumArgs a) {
  __shared__ float4 sums[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x;
  const int c = blockIdx.y * kJoinCols + lane * 4;
  const int64_t begin = static_cast<int64_t>(i) * a.per_block, end = begin + a.per_block;
  const uint32_t key = a.sorted[end - 1].x;
  const uint32_t next = a.sorted[end].x;
  const uint32_t before = begin > 0 ? a.sorted[begin - 1].x : a.rows;
  if (key == static_cast<uint32_t>(a.rows) || next != key || before == key) return;
  // the first sorted token past the run
  int64_t lo = end + 1, hi = a.T;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (a.sorted[mid].x == key)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int to = static_cast<int>((lo - 1) / a.per_block);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < a.Dp) {
#pragma unroll 4
    for (int m = i + warp; m <= to; m += kJoinWarps) {
      const float4 p = *reinterpret_cast<const float4*>(
          a.part + (static_cast<int64_t>(m) * 2 + (m == i ? 1 : 0)) * a.Dp + c);
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kJoinWarps; ++w) {
      const float4 p = sums[w][lane];
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float one[1] = {v[e]};
      if (c + e < a.D) put_row<1>(a, key, c + e, one);
    }
  }
}

// The sums, then the runs that cross blocks. Launched kernels are added to n.
template <class In, int VEC, int G>
cudaError_t run_sum(SumArgs a, int& n, cudaStream_t stream) {
  a.windows = (a.D + G * VEC - 1) / (G * VEC);
  a.per_block = a.chunk * (kSumThreads / G);
  a.nblocks = static_cast<int>((static_cast<int64_t>(a.T) + a.per_block - 1) / a.per_block);
  const int64_t blocks = static_cast<int64_t>(a.nblocks) * a.windows;
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
  sum_kernel<In, VEC, G><<<static_cast<unsigned>(blocks), kSumThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++n;
  if (a.nblocks > 1) {
    const dim3 grid(a.nblocks - 1, (a.D + kJoinCols - 1) / kJoinCols);
    if (grid.y > 65535) return cudaErrorInvalidValue;
    join_kernel<<<grid, kJoinWarps * 32, 0, stream>>>(a);
    e = cudaGetLastError();
    ++n;
  }
  return e;
}

template <class In>
cudaError_t run_sum_shape(const SumArgs& a, bool vec, int& n, cudaStream_t stream) {
  constexpr int V = kVecOf<In>;
  if (!vec) return run_sum<In, 1, 32>(a, n, stream);
  const int chunks = a.D / V;
  if (chunks <= 4) return run_sum<In, V, 4>(a, n, stream);
  if (chunks <= 8) return run_sum<In, V, 8>(a, n, stream);
  if (chunks <= 16) return run_sum<In, V, 16>(a, n, stream);
  return run_sum<In, V, 32>(a, n, stream);
}

// Sizes of a gradient's scratch, and where its parts lie.
struct GradPlan {
  int sort_blocks, per, passes, bits;
  int chunk;
  int64_t nblocks, Dp;
  int64_t pairs[2], counts, part, bytes;  // byte offsets, and the sum
};

GradPlan plan_grad(int64_t T, int64_t rows, int64_t D) {
  GradPlan p;
  int key_bits = 0;  // of the largest key, `rows`
  while ((rows >> key_bits) != 0) ++key_bits;
  p.passes = (key_bits + 7) / 8;
  p.bits = (key_bits + p.passes - 1) / p.passes;
  int64_t per = (T + kSortMaxBlocks - 1) / kSortMaxBlocks;
  per = std::max<int64_t>(1, (per + kSortThreads - 1) / kSortThreads) * kSortThreads;
  p.per = static_cast<int>(per);
  p.sort_blocks = static_cast<int>((T + per - 1) / per);
  // a group's tokens: as few as are in flight at once while that fills the
  // GPU's threads, more when there are more; by T and D alone
  const int64_t even = T * D / (int64_t{148} * 1024 * 4) / kSumInFlight * kSumInFlight;
  p.chunk = static_cast<int>(std::min<int64_t>(256, std::max<int64_t>(kSumInFlight, even)));
  // blocks of chunks, at most: 32 lanes a group are the widest
  const int64_t per_block = static_cast<int64_t>(p.chunk) * (kSumThreads / 32);
  p.nblocks = (T + per_block - 1) / per_block;
  p.Dp = (D + 7) / 8 * 8;
  int64_t at = 0;
  auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.pairs[0] = take(T * 8);
  p.pairs[1] = take(T * 8);
  p.counts = take(static_cast<int64_t>(p.sort_blocks) * kRadix * 4);
  p.part = take(p.nblocks * 2 * p.Dp * 4);
  p.bytes = at;
  return p;
}

bool grad_sizes_ok(int64_t T, int64_t rows, int64_t D) {
  return T >= 0 && T <= INT_MAX && rows >= 1 && rows <= INT_MAX - 1 && D >= 1 &&
         D <= (1 << 22);
}

int clear_status(int32_t* status, cudaStream_t stream) {
  if (status == nullptr) return DLRM_OK;
  const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), stream);
  return e == cudaSuccess ? DLRM_OK : cuda_fail(e);
}

}  // namespace
}  // namespace dlrm

extern "C" {

int dlrm_embedding_lookup(const void* table, int table_dtype, int64_t ldw, int64_t rows,
                          int64_t D, const int32_t* ids, int64_t T, float scale,
                          int64_t padding_idx, void* out, int out_dtype, int64_t ldo,
                          int32_t* status_dev, dlrm_stream_t stream) {
  using namespace dlrm;
  if (!known_dtype(table_dtype) || !known_dtype(out_dtype)) return DLRM_ERR_ARG;
  if (!grad_sizes_ok(T, rows, D) || ldw < D || ldo < D) return DLRM_ERR_SHAPE;
  if (padding_idx < -1 || padding_idx >= rows) return DLRM_ERR_ARG;
  if (T > 0 && (table == nullptr || ids == nullptr || out == nullptr)) return DLRM_ERR_NULL;
  const int es = dtype_size(table_dtype), os = dtype_size(out_dtype);
  if (!is_aligned(table, es) || !is_aligned(out, os) || !is_aligned(ids, 4) ||
      !is_aligned(status_dev, 4))
    return DLRM_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = clear_status(status_dev, s);
  if (rc != DLRM_OK || T == 0) return rc;
  LookupArgs a = {};
  a.table = table;
  a.ldw = ldw;
  a.ids = ids;
  a.out = out;
  a.ldo = ldo;
  a.rows = static_cast<int>(rows);
  a.D = static_cast<int>(D);
  a.T = static_cast<int>(T);
  a.pad = static_cast<int>(padding_idx);
  a.scale = scale;
  a.status = status_dev;
  const bool vec = D % (16 / es) == 0 && rows16(table, ldw, es) && rows16(out, ldo, os);
  using B = __nv_bfloat16;
  cudaError_t e;
  if (table_dtype == DLRM_TABLE_F32)
    e = out_dtype == DLRM_TABLE_F32 ? run_lookup_shape<float, float>(a, vec, s)
                                    : run_lookup_shape<float, B>(a, vec, s);
  else
    e = out_dtype == DLRM_TABLE_F32 ? run_lookup_shape<B, float>(a, vec, s)
                                    : run_lookup_shape<B, B>(a, vec, s);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

int64_t dlrm_embedding_grad_scratch_bytes(int64_t T, int64_t rows, int64_t D) {
  using namespace dlrm;
  if (!grad_sizes_ok(T, rows, D)) return DLRM_ERR_SHAPE;
  return plan_grad(T, rows, D).bytes;
}

int dlrm_embedding_grad(const void* grad, int grad_dtype, int64_t ldg, const int32_t* ids,
                        int64_t T, int64_t L, int64_t rows, int64_t D, float scale,
                        int64_t padding_idx, void* out, int out_dtype, int64_t ldo,
                        int accumulate, void* scratch, int64_t scratch_bytes,
                        int32_t* status_dev, dlrm_stream_t stream) {
  using namespace dlrm;
  if (!known_dtype(grad_dtype) || !known_dtype(out_dtype)) return DLRM_ERR_ARG;
  if (!grad_sizes_ok(T, rows, D) || ldg < D || ldo < D || L < 1 || T % L != 0)
    return DLRM_ERR_SHAPE;
  if (padding_idx < -1 || padding_idx >= rows) return DLRM_ERR_ARG;
  if (out == nullptr || (T > 0 && (grad == nullptr || ids == nullptr))) return DLRM_ERR_NULL;
  const int es = dtype_size(grad_dtype), os = dtype_size(out_dtype);
  if (!is_aligned(grad, es) || !is_aligned(out, os) || !is_aligned(ids, 4) ||
      !is_aligned(status_dev, 4) || !is_aligned(scratch, 16))
    return DLRM_ERR_ALIGN;
  const GradPlan p = plan_grad(T, rows, D);
  if (scratch_bytes < p.bytes) return DLRM_ERR_SCRATCH;
  if (T > 0 && scratch == nullptr) return DLRM_ERR_NULL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = clear_status(status_dev, s);
  if (rc != DLRM_OK) return rc;
  if (!accumulate) {
    const cudaError_t e = cudaMemset2DAsync(out, static_cast<size_t>(ldo) * os, 0,
                                            static_cast<size_t>(D) * os, rows, s);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  if (T == 0) return DLRM_OK;

  char* mem = static_cast<char*>(scratch);
  SortArgs sa = {};
  sa.ids = ids;
  sa.counts = reinterpret_cast<uint32_t*>(mem + p.counts);
  sa.T = static_cast<int>(T);
  sa.rows = static_cast<int>(rows);
  sa.pad = static_cast<int>(padding_idx);
  sa.bits = p.bits;
  sa.per = p.per;
  sa.status = status_dev;
  for (int i = 0; i < p.passes; ++i) {
    sa.out = reinterpret_cast<uint2*>(mem + p.pairs[i & 1]);
    sa.shift = i * p.bits;
    sort_count_kernel<<<p.sort_blocks, kSortThreads, 0, s>>>(sa);
    sort_move_kernel<<<p.sort_blocks, kSortThreads, 0, s>>>(sa);
    sa.ids = nullptr;
    sa.in = sa.out;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);

  SumArgs a = {};
  a.grad = grad;
  a.ldg = ldg;
  a.sorted = sa.out;
  a.part = reinterpret_cast<float*>(mem + p.part);
  a.Dp = p.Dp;
  a.out = out;
  a.ldo = ldo;
  a.T = static_cast<int>(T);
  a.L = static_cast<int>(L);
  a.rows = static_cast<int>(rows);
  a.D = static_cast<int>(D);
  a.chunk = p.chunk;
  a.scale = scale;
  a.out_bf16 = out_dtype == DLRM_TABLE_BF16;
  a.accumulate = accumulate ? 1 : 0;
  const bool vec = D % (16 / es) == 0 && rows16(grad, ldg, es) && rows16(out, ldo, os);
  int n = 2 * p.passes;
  e = grad_dtype == DLRM_TABLE_F32 ? run_sum_shape<float>(a, vec, n, s)
                                   : run_sum_shape<__nv_bfloat16>(a, vec, n, s);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch(n);
  return DLRM_OK;
}

}  // extern "C"
