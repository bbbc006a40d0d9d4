// Embedding rows by token id, and the table's gradient by sorted tokens
// (declared in dlrm_tokens.h).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstddef>

#include "common.h"
#include "dlrm_tokens.h"
#include "tma_common.cuh"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxDevices = 64;  // devices whose launch set-up is cached

// ---------------------------------------------------------------------------
// Lookup: Y[t] = scale * W[ids[t]].
//
// G lanes take a window of G * E * VEC columns of kRowsInFlight tokens' rows, all
// loads in the air before the first is used. No arithmetic to speak of: bound by
// the bytes of the rows, or, where 128-bit accesses cannot walk them, by the number
// of accesses. Y is written past the cache's order of use, which keeps frequent
// rows in L2. Measured on B200, 1310720 tokens of 512-byte rows under a power law
// of 1.2 (671 MB written): 119 to 125 us over several GPUs, of 2000-byte rows, 16383
// tokens: 10.2 us (6.4 TB/s), 15.8 where a group walks all windows of its rows. More
// threads a block (256, 512) cost 6 and 13 us of the first, two rows in flight 12,
// ordinary stores 4. 60000 rows of 1001 f32, single elements: 76 us with four
// accesses a lane (6.3 TB/s), bf16 58; of 1002, pairs: 74 and 41.

constexpr int kLookupThreads = 128;
constexpr int kRowsInFlight = 4;

struct LookupArgs {
  const void* table;
  int64_t ldw;
  const int32_t* ids;
  void* out;
  int64_t ldo;
  int rows, D, T, pad;
  int windows;  // of G * VEC columns
  float scale;
  int32_t* status;
};

template <class In, class Out, int VEC, int G, int E>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const LookupArgs a) {
  const In* W = static_cast<const In*>(a.table);
  Out* Y = static_cast<Out*>(a.out);
  const int q = threadIdx.x % G;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x) / G;
  const int64_t t0 = unit / a.windows * kRowsInFlight;
  const int c0 = (static_cast<int>(unit % a.windows) * G * E + q) * VEC;
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
  Raw<In, VEC> raw[kRowsInFlight][E];
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    const In* row = W + static_cast<int64_t>(id[u]) * a.ldw + c0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      raw[u][e] = Raw<In, VEC>();
      if (id[u] >= 0 && id[u] < a.rows && c0 + e * G * VEC < a.D)
        raw[u][e] = __ldg(reinterpret_cast<const Raw<In, VEC>*>(row + e * G * VEC));
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsInFlight; ++u) {
    Out* row = Y + (t0 + u) * a.ldo + c0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v[VEC];
      widen<In, VEC>(raw[u][e], v);
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[k] = id[u] < a.rows ? v[k] * a.scale : 0.f;
      if (id[u] >= 0 && c0 + e * G * VEC < a.D)
        store_f32<Out, VEC, true>(row + e * G * VEC, v);
    }
  }
}

// The lanes of a group, and the accesses of a lane (E of them, G apart), by the
// row's length: 128-bit accesses where rows allow them, else VEC = 2 or 1 elements
// and more accesses a lane.
template <class In, int VEC, class F>
cudaError_t by_narrow(int chunks, F& f) {
  if (chunks <= 16) return f.template run<In, VEC, 8, 2>();
  if (chunks <= 32) return f.template run<In, VEC, 8, 4>();
  if (chunks <= 64) return f.template run<In, VEC, 16, 4>();
  if (chunks > 128 && chunks <= 256) return f.template run<In, VEC, 32, 8>();
  return f.template run<In, VEC, 32, 4>();
}

template <class In, class F>
cudaError_t by_shape(int D, int vec, F& f) {
  constexpr int V = kVecOf<In>;
  const int chunks = D / vec;
  if (vec == 1) return by_narrow<In, 1>(chunks, f);
  if (vec == 2) return by_narrow<In, 2>(chunks, f);
  if (chunks <= 4) return f.template run<In, V, 4, 1>();
  if (chunks <= 8) return f.template run<In, V, 8, 1>();
  if (chunks <= 16) return f.template run<In, V, 16, 1>();
  return f.template run<In, V, 32, 1>();
}

template <class F>
cudaError_t by_type(int dtype, int D, int vec, F& f) {
  return dtype == DLRM_TABLE_F32 ? by_shape<float>(D, vec, f)
                                 : by_shape<__nv_bfloat16>(D, vec, f);
}

// Elements of an access that both matrices' rows allow.
int common_vec(const void* in, int64_t ldi, int in_size, const void* out, int64_t ldo,
               int out_size, int64_t D) {
  for (int v : {16 / in_size, 2})
    if (D % v == 0 && rows_by(in, ldi, in_size, v) && rows_by(out, ldo, out_size, v)) return v;
  return 1;
}

template <class Out>
struct LookupLaunch {
  LookupArgs a;
  cudaStream_t stream;
  template <class In, int VEC, int G, int E>
  cudaError_t run() {
    constexpr int kWindow = G * E * VEC;
    a.windows = (a.D + kWindow - 1) / kWindow;
    const int64_t units =
        (static_cast<int64_t>(a.T) + kRowsInFlight - 1) / kRowsInFlight * a.windows;
    const int64_t blocks = (units * G + kLookupThreads - 1) / kLookupThreads;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    return launch(&lookup_kernel<In, Out, VEC, G, E>, dim3(static_cast<unsigned>(blocks)),
                  kLookupThreads, 0, false, stream, a);
  }
};

// ---------------------------------------------------------------------------
// Gradient: zeros for the rows that no token names.
//
// A dense gradient is mostly writes, and the sort in front of the sums leaves
// the memory idle; so every row is zeroed while the tokens are sorted (by a warp
// of the sort's own blocks, or a kernel beside it), and the named rows are
// written over later.

struct FillArgs {
  char* out;      // null: nothing to fill
  int64_t rows;   // of row_bytes each, pitch bytes apart
  int64_t row_bytes, pitch;
  int unit;  // bytes of the widest store that every row allows: 16, 8, 4 or 2

  bool apart() const { return pitch != row_bytes; }
};

__device__ __forceinline__ void put_zeros(char* p, int unit) {
  if (unit == 16)
    *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
  else if (unit == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(0, 0);
  else if (unit == 4)
    *reinterpret_cast<uint32_t*>(p) = 0;
  else
    *reinterpret_cast<uint16_t*>(p) = 0;
}

// Bulk (TMA, non-tensor) copy of `bytes` bytes of this CTA's shared memory (a
// multiple of 16; both addresses 16-byte aligned) to global memory, tracked by
// the thread's bulk groups.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

constexpr int kZeroBytes = 16 << 10;  // of a bulk store

// Parts part, part + apart, .. (`count` of them) of `parts` of the zeros of rows without
// gaps, by one whole warp: bulk stores of a block of zeros, which one lane issues; it
// waits where the SM's queue of them is full, so the warp has nothing else to do
// meanwhile. zeros: kZeroBytes of shared memory, 16-byte aligned, for this alone. The
// warp has to call fill_done before it ends.
__device__ void fill_zeros(const FillArgs& f, int part, int parts, uint8_t* zeros, int count = 1,
                           int apart = 0) {
  const int lane = threadIdx.x & 31;
  const int64_t bytes = f.rows * f.row_bytes;
  const int64_t lead = min(bytes, static_cast<int64_t>(-reinterpret_cast<intptr_t>(f.out) & 15));
  const int64_t mid = (bytes - lead) & ~int64_t{15};
  for (int i = lane; i < kZeroBytes / 16; i += 32)
    reinterpret_cast<uint4*>(zeros)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    for (int k = 0; k < count; ++k)
      for (int64_t at = static_cast<int64_t>(part + k * apart) * kZeroBytes; at < mid;
           at += static_cast<int64_t>(parts) * kZeroBytes)
        bulk_s2g(f.out + lead + at, zeros,
                 static_cast<uint32_t>(min(static_cast<int64_t>(kZeroBytes), mid - at)));
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
  if (part == 0) {  // the unaligned ends
    if (lane < lead) f.out[lane] = 0;
    if (lane < bytes - lead - mid) f.out[lead + mid + lane] = 0;
  }
}

// The zeros that this warp began are written.
__device__ __forceinline__ void fill_done() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The zeros alone, behind a cluster sort and at the same time: a block for each
// SM that the sort leaves. An SM writes about 60 GB/s of bulk stores however
// many blocks share it, so the blocks must not: each asks for half of the shared
// memory. 256 MB take 40 us so, the memory's rate; with 148 small blocks, some
// of them two on an SM, 59 us, where most had ended after 32. (Fill blocks in
// clusters of the sort's own launch took 41 or 45 us, by how many clusters the
// GPU at hand keeps resident.)
constexpr int kFillThreads = 32;
constexpr int kFillSmem = 116 << 10;

// BESIDE: the sums follow, and their blocks may be scheduled early (they wait for this
// grid's end; what follows zeros alone may not).
template <bool BESIDE>
__global__ void __launch_bounds__(kFillThreads) fill_kernel(const FillArgs f) {
  extern __shared__ __align__(16) uint8_t zeros[];
  static_assert(kFillSmem >= kZeroBytes, "room for the zeros");
  if constexpr (BESIDE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  fill_zeros(f, blockIdx.x, gridDim.x, zeros);
  fill_done();
  // The sort in front is still at work, perhaps: this grid ends after it, so that
  // what waits for the zeros has the sorted tokens too.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The zeros of rows that lie apart from each other (columns of a wider buffer): ordinary
// stores, `lanes` of them a row at a time, by whole blocks; beside a cluster sort as
// above, or in front of a longer one. (By the sort's warps and two bytes at a time, an
// earlier form, a million rows of 64 f32 with gaps took 800 us of a gradient.)
constexpr int kFillRowThreads = 256;

template <bool BESIDE>
__global__ void __launch_bounds__(kFillRowThreads) fill_rows_kernel(const FillArgs f, int lanes) {
  if constexpr (BESIDE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t per_row = f.row_bytes / f.unit;
  const int at = threadIdx.x / lanes, step = kFillRowThreads / lanes;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * step + at; r < f.rows;
       r += static_cast<int64_t>(gridDim.x) * step)
    for (int64_t c = threadIdx.x % lanes; c < per_row; c += lanes)
      put_zeros(f.out + r * f.pitch + c * f.unit, f.unit);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as above
}

// ---------------------------------------------------------------------------
// Gradient, step 1: the tokens sorted by id, stable.
//
// Least-significant-digit radix sort of (key, token) pairs with digits of at
// most 8 bits over the bits that `rows` needs. Padding and out-of-range ids
// take the key `rows` and so come last. Up to kClusterSort tokens one cluster
// of CTAs sorts in shared memory, all passes in one launch; more take two
// launches a pass: every block counts the digits of its stretch of pairs, then
// every block adds up the counts of all digits and of the blocks before it,
// and moves its pairs. Either way a block first brings a tile of pairs into
// digit order in its own shared memory, so that neighbouring threads write
// neighbouring places: moving the pairs straight from registers, a store of
// scattered 8-byte pairs a warp, took 1.5 us a pair of a thread and pass.

constexpr int kRadix = 256;
constexpr int kSortThreads = 512;  // of a block that counts or moves
constexpr int kSortItems = 16;     // pairs of a thread, at most, in a tile
constexpr int kSortMaxBlocks = 2 * kSms;
// A move takes more than twice as long as a count (19 and 8 us at 1.3 M pairs) and
// writes more of the zeros meanwhile: 512 MB of them, in all 271 us with equal
// parts, 263 with two of three in the moves, 258 with three of four.
constexpr int kMoveParts = 3, kPassParts = kMoveParts + 1;
constexpr int kClusterThreads = 1024;
constexpr int kClusterSize = 8;       // CTAs
constexpr int kClusterMaxItems = 8;  // pairs of a thread
constexpr int64_t kClusterSort = int64_t{kClusterSize} * kClusterThreads * kClusterMaxItems;

struct SortArgs {
  const int32_t* ids;  // first pass: the tokens' ids; later passes read `in`
  const uint2* in;     // (key, token)
  uint2* out;
  uint32_t* counts;  // [block][kRadix]
  int T, rows, pad;
  int shift, bits;
  int passes;  // of the cluster sort
  int per;     // pairs of a block, a multiple of its tile
  int blocks;  // that sort; the grid may have more, which only fill
  FillArgs fill;
  int fill_part, fill_parts;  // the first block's part of the zeros, and of how many
  int32_t* status;
};

__device__ __forceinline__ uint2 sort_pair(const SortArgs& a, int64_t i) {
  if (a.ids == nullptr) return a.in[i];
  const int r = __ldg(a.ids + i);
  const bool in = static_cast<unsigned>(r) < static_cast<unsigned>(a.rows);
  const uint32_t key = (in && r != a.pad) ? r : a.rows;
  return make_uint2(key, static_cast<uint32_t>(i));
}

__device__ __forceinline__ void flag_bad_id(const SortArgs& a, int64_t i) {
  if (a.ids != nullptr && a.status != nullptr &&
      static_cast<unsigned>(__ldg(a.ids + i)) >= static_cast<unsigned>(a.rows))
    atomicOr(a.status, DLRM_FLAG_INDEX_OOB);
}

// The live lanes of the warp whose digit is this lane's (for a live lane): a vote
// for each of the digit's bits. (The match instruction takes the warp's
// distinct digits one after another.)
__device__ __forceinline__ unsigned same_digit(uint32_t digit, bool live, int bits) {
  unsigned peers = __ballot_sync(kFull, live);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    if (b < bits) {
      const bool set = (digit >> b) & 1;
      const unsigned votes = __ballot_sync(kFull, set);
      peers &= set ? votes : ~votes;
    }
  }
  return peers;
}

// A barrier of the THREADS threads that sort (a warp more may be filling).
template <int THREADS>
__device__ __forceinline__ void sort_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Exclusive sums over the digits, for the threads below kRadix; every thread that
// sorts takes part. Holds a barrier.
template <int THREADS>
__device__ __forceinline__ uint32_t digits_before(uint32_t n, uint32_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t scan = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t m = __shfl_up_sync(kFull, scan, o);
    if (lane >= o) scan += m;
  }
  if (threadIdx.x < kRadix && lane == 31) warp_sum[warp] = scan;
  sort_sync<THREADS>();
  if (threadIdx.x < kRadix)
    for (int w = 0; w < warp; ++w) scan += warp_sum[w];
  return scan - n;
}

template <int THREADS, int ITEMS>
struct TileSmem {
  static constexpr int kWarps = THREADS / 32;
  static constexpr int kParts = THREADS / kRadix;  // threads of a digit
  static constexpr int kWarpsOfPart = kWarps / kParts;
  alignas(16) uint2 pairs[THREADS * ITEMS];  // the tile in digit order
  uint32_t at[kWarps][kRadix];
  uint32_t parts[kParts][kRadix];
  uint32_t start[kRadix];  // a digit's first place in `pairs`
  uint32_t warp_sum[kRadix / 32];
};

// Brings a tile of pairs (a warp's ITEMS * 32 pairs follow each other, `n` of the
// tile are live) into digit order in sm.pairs, stable. Returns the count of
// digit threadIdx.x for the threads below kRadix. Ends with a barrier.
template <int THREADS, int ITEMS>
__device__ __forceinline__ uint32_t order_tile(TileSmem<THREADS, ITEMS>& sm,
                                               const uint2 (&pair)[ITEMS], int n, int shift,
                                               int bits) {
  using S = TileSmem<THREADS, ITEMS>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int own = warp * 32 * ITEMS + lane;
  const uint32_t mask = (1u << bits) - 1;
  // a pair's place among its warp's pairs of the same digit
  uint32_t among[ITEMS];
#pragma unroll
  for (int d = lane; d < kRadix; d += 32) sm.at[warp][d] = 0;
  __syncwarp();
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    const bool live = own + u * 32 < n;
    const uint32_t digit = (pair[u].x >> shift) & mask;
    const unsigned peers = same_digit(digit, live, bits);
    among[u] = live ? sm.at[warp][digit] + __popc(peers & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (live && lane == __ffs(peers) - 1) sm.at[warp][digit] += __popc(peers);
    __syncwarp();
  }
  sort_sync<THREADS>();
  // ... among the tile's warps: kWarpsOfPart of them a thread, then the threads of a digit
  const int d = tid % kRadix, part = tid / kRadix;
  uint32_t sum = 0;
#pragma unroll
  for (int w = 0; w < S::kWarpsOfPart; ++w) {
    uint32_t& c = sm.at[part * S::kWarpsOfPart + w][d];
    const uint32_t m = c;
    c = sum;
    sum += m;
  }
  sm.parts[part][d] = sum;
  sort_sync<THREADS>();
  uint32_t count = 0;
#pragma unroll
  for (int k = 0; k < S::kParts; ++k) count += sm.parts[k][d];
  // ... and after the smaller digits
  uint32_t place = digits_before<THREADS>(count, sm.warp_sum);
  if (part == 0) {
    sm.start[d] = place;
#pragma unroll
    for (int k = 0; k < S::kParts; ++k) {
      const uint32_t m = sm.parts[k][d];
      sm.parts[k][d] = place;
      place += m;
    }
  }
  sort_sync<THREADS>();
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    if (own + u * 32 < n) {
      const uint32_t digit = (pair[u].x >> shift) & mask;
      sm.pairs[sm.parts[warp / S::kWarpsOfPart][digit] + sm.at[warp][digit] + among[u]] = pair[u];
    }
  }
  sort_sync<THREADS>();
  return count;
}

__global__ void __launch_bounds__(kSortThreads + 32, 2) sort_count_kernel(const SortArgs a) {
  __shared__ __align__(16) uint8_t zeros[kZeroBytes];
  __shared__ uint32_t cnt[kRadix];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pass before is done
  if (tid >= kSortThreads) {
    fill_zeros(a.fill, a.fill_part + blockIdx.x, a.fill_parts, zeros);
    fill_done();
    return;
  }
  if (static_cast<int>(blockIdx.x) >= a.blocks) return;
  if (tid < kRadix) cnt[tid] = 0;
  sort_sync<kSortThreads>();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.per;
  const int64_t end = min(begin + a.per, static_cast<int64_t>(a.T));
  const uint32_t mask = (1u << a.bits) - 1;
  constexpr int kLoads = 4;  // pairs a thread loads at once
  for (int64_t i0 = begin; i0 < end; i0 += kSortThreads * kLoads) {
    uint32_t digit[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int64_t i = i0 + u * kSortThreads + tid;
      digit[u] = kRadix;  // of no pair
      if (i < end) {
        flag_bad_id(a, i);
        digit[u] = (sort_pair(a, i).x >> a.shift) & mask;
      }
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      // a warp whose digits are all the same (one frequent id) adds once
      const bool same = __all_sync(kFull, digit[u] == __shfl_sync(kFull, digit[u], 0));
      if (digit[u] != kRadix && (!same || (tid & 31) == 0))
        atomicAdd(&cnt[digit[u]], same ? 32 : 1);
    }
  }
  sort_sync<kSortThreads>();
  if (tid < kRadix) a.counts[static_cast<int64_t>(blockIdx.x) * kRadix + tid] = cnt[tid];
}

template <int ITEMS>
struct MoveSmem {
  TileSmem<kSortThreads, ITEMS> tile;
  uint8_t zeros[kZeroBytes];
  uint32_t place[kRadix];  // a digit's next place in the output
};

template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads + 32, 2) sort_move_kernel(const SortArgs a) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  auto& sm = *reinterpret_cast<MoveSmem<ITEMS>*>(sort_smem);
  static_assert(offsetof(MoveSmem<ITEMS>, zeros) % 16 == 0, "bulk stores");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts are there
  if (threadIdx.x >= kSortThreads) {
    fill_zeros(a.fill, a.fill_part + blockIdx.x, a.fill_parts, sm.zeros, kMoveParts, gridDim.x);
    fill_done();
    return;
  }
  if (static_cast<int>(blockIdx.x) < a.blocks) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t mask = (1u << a.bits) - 1;
    constexpr int kTile = kSortThreads * ITEMS;
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.per;
    const int64_t end = min(begin + a.per, static_cast<int64_t>(a.T));
    uint2 pair[ITEMS];
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int u = 0; u < ITEMS; ++u) {
        const int64_t i = i0 + (warp * ITEMS + u) * 32 + lane;
        pair[u] = make_uint2(0, 0);
        if (i < end) pair[u] = sort_pair(a, i);
      }
    };
    load(begin);
    // pairs of each digit in all blocks and in the blocks before this one: four
    // digits a thread, every eighth block
    {
      const int d4 = tid % (kRadix / 4), part = tid / (kRadix / 4);
      const uint4* counts = reinterpret_cast<const uint4*>(a.counts) + d4;
      uint4 all = make_uint4(0, 0, 0, 0), mine = all;
#pragma unroll 8
      for (int b = part; b < a.blocks; b += 8) {
        const uint4 c = counts[static_cast<int64_t>(b) * (kRadix / 4)];
        all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
        if (b < static_cast<int>(blockIdx.x))
          mine.x += c.x, mine.y += c.y, mine.z += c.z, mine.w += c.w;
      }
      // the tile's pairs come later
      static_assert(sizeof(sm.tile.pairs) >= 2 * 8 * kRadix * 4, "room for the sums");
      uint4* sums = reinterpret_cast<uint4*>(sm.tile.pairs);
      sums[part * (kRadix / 4) + d4] = all;
      sums[(8 + part) * (kRadix / 4) + d4] = mine;
    }
    sort_sync<kSortThreads>();
    uint32_t all = 0, place = 0;
    if (tid < kRadix) {
      const uint32_t* sums = reinterpret_cast<const uint32_t*>(sm.tile.pairs);
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        all += sums[p * kRadix + tid];
        place += sums[(8 + p) * kRadix + tid];
      }
    }
    place += digits_before<kSortThreads>(all, sm.tile.warp_sum);
    if (tid < kRadix) sm.place[tid] = place;
    for (int64_t i0 = begin; i0 < end; i0 += kTile) {
      const int n = static_cast<int>(min(static_cast<int64_t>(kTile), end - i0));
      if (i0 > begin) load(i0);
      sort_sync<kSortThreads>();  // the tile before has left, its digits' places are set
      const uint32_t count = order_tile(sm.tile, pair, n, a.shift, a.bits);
#pragma unroll 4
      for (int k = tid; k < n; k += kSortThreads) {
        const uint2 p = sm.tile.pairs[k];
        const uint32_t digit = (p.x >> a.shift) & mask;
        a.out[sm.place[digit] + (k - sm.tile.start[digit])] = p;
      }
      sort_sync<kSortThreads>();
      if (tid < kRadix) sm.place[tid] += count;
    }
  }
}

__device__ __forceinline__ uint32_t load_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_cluster_pair(uint32_t cluster_addr, uint2 p) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(cluster_addr), "r"(p.x), "r"(p.y)
               : "memory");
}

template <int ITEMS>
struct ClusterSmem {
  TileSmem<kClusterThreads, ITEMS> tile;
  uint2 arrived[kClusterThreads * ITEMS];  // this CTA's stretch of the pairs after a pass
  uint32_t total[kRadix];                  // its count of each digit, read by the others
  uint32_t place[kRadix];
  alignas(16) uint8_t zeros[kZeroBytes];
};

// One cluster sorts: each of its CTAs owns a stretch of the pairs, a tile. Few
// zeros it writes itself.
template <int ITEMS>
__global__ void __launch_bounds__(kClusterThreads, 1) sort_cluster_kernel(const SortArgs a) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  // the fill's or the sums' blocks may be scheduled now: these wait for this
  // grid's end, those have nothing to do with it before theirs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto& sm = *reinterpret_cast<ClusterSmem<ITEMS>*>(sort_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  constexpr int kStretch = kClusterThreads * ITEMS;
  const int own = warp * 32 * ITEMS + lane;  // the thread's first pair in the stretch
  const int n = max(0, min(kStretch, a.T - rank * kStretch));
  const uint32_t mask = (1u << a.bits) - 1;
  uint2 pair[ITEMS];
#pragma unroll
  for (int u = 0; u < ITEMS; ++u) {
    pair[u] = make_uint2(0, 0);
    if (own + u * 32 < n) {
      pair[u] = sort_pair(a, rank * kStretch + own + u * 32);
      flag_bad_id(a, rank * kStretch + own + u * 32);
    }
  }
  if (a.fill.out != nullptr && warp == 0) fill_zeros(a.fill, rank, kClusterSize, sm.zeros);
  for (int p = 0; p < a.passes; ++p) {
    const int shift = p * a.bits;
    const uint32_t count = order_tile(sm.tile, pair, n, shift, a.bits);
    if (tid < kRadix) sm.total[tid] = count;
    cluster_sync();
    // a digit's first place: after the smaller digits, and after the CTAs before
    uint32_t all = 0, place = 0;
    if (tid < kRadix) {
      const uint32_t addr = smem_u32(&sm.total[tid]);
#pragma unroll
      for (int r = 0; r < kClusterSize; ++r) {
        const uint32_t c = load_cluster_u32(map_to_cta(addr, r));
        all += c;
        place += r < rank ? c : 0;
      }
    }
    place += digits_before<kClusterThreads>(all, sm.tile.warp_sum);
    if (tid < kRadix) sm.place[tid] = place;
    __syncthreads();
    const bool final_pass = p + 1 == a.passes;
    for (int k = tid; k < n; k += kClusterThreads) {
      const uint2 v = sm.tile.pairs[k];
      const uint32_t digit = (v.x >> shift) & mask;
      const uint32_t to = sm.place[digit] + (k - sm.tile.start[digit]);
      if (final_pass)
        a.out[to] = v;
      else
        store_cluster_pair(map_to_cta(smem_u32(&sm.arrived[to % kStretch]), to / kStretch), v);
    }
    // the pairs have arrived, and nobody reads this CTA's counts any more
    cluster_sync();
    if (!final_pass) {
#pragma unroll
      for (int u = 0; u < ITEMS; ++u) pair[u] = sm.arrived[own + u * 32];
    }
  }
  if (a.fill.out != nullptr && warp == 0) fill_done();
}

// A kernel's dynamic shared memory, set once per device (`prepared` is its own).
template <class K>
cudaError_t allow_smem(K* fn, int bytes, std::atomic<bool> (&prepared)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cacheable = dev >= 0 && dev < kMaxDevices;
  if (cacheable && prepared[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && cacheable) prepared[dev].store(true, std::memory_order_release);
  return e;
}

// The zeros: beside the cluster sort that was launched last (the one before them
// that they may not wait for), or behind all that is on the stream. blocks: SMs to take.
template <bool BESIDE>
cudaError_t run_fill(const FillArgs& f, int blocks, cudaStream_t stream) {
  if (f.apart()) {
    int lanes = 1;  // a power of two
    while (lanes < 32 && lanes < f.row_bytes / f.unit) lanes *= 2;
    return launch(&fill_rows_kernel<BESIDE>, dim3(blocks * (2048 / kFillRowThreads)),
                  kFillRowThreads, 0, BESIDE, stream, f, lanes);
  }
  static std::atomic<bool> prepared[kMaxDevices];
  const cudaError_t e = allow_smem(&fill_kernel<BESIDE>, kFillSmem, prepared);
  if (e != cudaSuccess) return e;
  return launch(&fill_kernel<BESIDE>, dim3(blocks), kFillThreads, kFillSmem, BESIDE, stream, f);
}

// Zeros that the cluster sort writes itself, 16 bulk stores a CTA; more go to a
// kernel beside it.
constexpr int64_t kClusterZeros = int64_t{kClusterSize} * 16 * kZeroBytes;

// Sorts up to kClusterSort tokens of `ids` into a.out and zeroes a.fill. Launched
// kernels are added to n.
template <int ITEMS>
cudaError_t run_cluster_sort(SortArgs& a, int sms, int& n, cudaStream_t stream) {
  auto* fn = &sort_cluster_kernel<ITEMS>;
  constexpr int smem = sizeof(ClusterSmem<ITEMS>);
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static std::atomic<bool> prepared[kMaxDevices];
  cudaError_t e = allow_smem(fn, smem, prepared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kClusterSize);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kClusterSize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const FillArgs fill = a.fill;
  const bool beside =
      fill.out != nullptr && (fill.apart() || fill.rows * fill.row_bytes > kClusterZeros);
  if (beside) a.fill.out = nullptr;
  ++n;
  if ((e = cudaLaunchKernelEx(&cfg, fn, a)) != cudaSuccess || !beside) return e;
  ++n;
  return run_fill<true>(fill, std::max(1, sms - kClusterSize), stream);
}

// Sorts more tokens, two launches a pass, between the two buffers of pairs; the
// zeros are shared out evenly over the launches. a.out ends as the sorted one.
template <int ITEMS>
cudaError_t run_grid_sort(SortArgs& a, uint2* const (&pairs)[2], cudaStream_t stream) {
  constexpr int smem = sizeof(MoveSmem<ITEMS>);
  auto* move = &sort_move_kernel<ITEMS>;
  static std::atomic<bool> prepared[kMaxDevices];
  cudaError_t e = allow_smem(move, smem, prepared);
  if (e != cudaSuccess) return e;
  // blocks enough to keep the memory busy with zeros
  const int grid = a.fill.out != nullptr ? std::max(a.blocks, kSms) : a.blocks;
  const int threads = a.fill.out != nullptr ? kSortThreads + 32 : kSortThreads;
  a.fill_parts = kPassParts * a.passes * grid;
  for (int i = 0; i < a.passes; ++i) {
    a.out = pairs[i & 1];
    a.shift = i * a.bits;
    a.fill_part = kPassParts * i * grid;
    // the first launch waits for all that came before it on the stream
    if ((e = launch(&sort_count_kernel, dim3(grid), threads, 0, i > 0, stream, a)) != cudaSuccess)
      return e;
    a.fill_part += grid;
    if ((e = launch(move, dim3(grid), threads, smem, true, stream, a)) != cudaSuccess) return e;
    a.ids = nullptr;
    a.in = a.out;
  }
  return cudaSuccess;
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

template <int VEC, int G, int E>
struct alignas(16) SumSmem {
  static constexpr int kGroups = kSumThreads / G;
  float head[kGroups][E][G * VEC];  // a group's part of a run that began before it
  uint32_t first[kGroups], last[kGroups];
};

// The block's sums over the sorted tokens [lo, hi), `chunk` of them a group (a
// multiple of kSumInFlight), for window `window` of the columns. part: this
// block's two rows for the runs that cross [lo, hi), or null if none does.
template <class In, int VEC, int G, int E>
__device__ __forceinline__ void sum_block(const SumArgs& a, SumSmem<VEC, G, E>& sm,
                                          const uint2* sorted, int64_t lo, int64_t hi, int chunk,
                                          int window, float* part) {
  constexpr int NG = SumSmem<VEC, G, E>::kGroups;
  // rows in flight: eight, or four of eight accesses a lane
  constexpr int U = G < kSumInFlight ? G : E >= 8 ? kSumInFlight / 2 : kSumInFlight;
  auto& first = sm.first;
  auto& last = sm.last;
  const int q = threadIdx.x % G, g = threadIdx.x / G, base = (threadIdx.x & 31) / G * G;
  const int c0 = (window * G * E + q) * VEC;  // the lane's columns: c0 + e * G * VEC ..
  auto live = [&](int e) { return c0 + e * G * VEC < a.D; };
  const int64_t begin = lo + static_cast<int64_t>(g) * chunk;
  const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(chunk), hi - begin)));
  const In* grad = static_cast<const In*>(a.grad);
  const uint32_t none = a.rows;
  const uint32_t left = (n > 0 && begin > 0) ? sorted[begin - 1].x : none;
  const uint32_t right = (n > 0 && begin + n < a.T) ? sorted[begin + n].x : none;
  if (q == 0) {
    first[g] = n > 0 ? sorted[begin].x : none;
    last[g] = n > 0 ? sorted[begin + n - 1].x : none;
  }
  float acc[E][VEC];
  auto clear = [&] {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[e][k] = 0.f;
  };
  auto keep_head = [&] {
#pragma unroll
    for (int e = 0; e < E; ++e) store_f32<float, VEC>(&sm.head[g][e][q * VEC], acc[e]);
  };
  auto add_head = [&](int j) {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[e][k] += sm.head[j][e][q * VEC + k];
  };
  auto put_rows = [&](uint32_t row) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (live(e)) put_row<VEC>(a, row, c0 + e * G * VEC, acc[e]);
  };
  auto put_part = [&](float* to) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (live(e)) store_f32<float, VEC>(to + c0 + e * G * VEC, acc[e]);
  };
  clear();
  uint32_t cur = none;  // key of the run being summed; none before the first
  bool inside = false;  // it began in this chunk
  // every lane of the warp takes the same number of steps: shuffles span it
  for (int j0 = 0; j0 < chunk; j0 += G) {
    uint32_t key = none, row = 0;
    if (j0 + q < n) {
      const uint2 p = sorted[begin + j0 + q];
      key = p.x;
      row = p.y / static_cast<uint32_t>(a.L);
    }
    const int steps = min(G, chunk - j0);
    for (int u0 = 0; u0 < steps; u0 += U) {
      Raw<In, VEC> raw[U][E];
      uint32_t k[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        k[u] = __shfl_sync(kFull, key, base + u0 + u);
        const uint32_t r = __shfl_sync(kFull, row, base + u0 + u);
        const In* from = grad + static_cast<int64_t>(r) * a.ldg + c0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          raw[u][e] = Raw<In, VEC>();
          if (k[u] != none && live(e))
            raw[u][e] = *reinterpret_cast<const Raw<In, VEC>*>(from + e * G * VEC);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k[u] != cur) {
          // the run before this token ends here
          if (cur != none) {
            if (!inside)
              keep_head();
            else
              put_rows(cur);
          }
          inside = k[u] != left || j0 + u0 + u > 0;
          cur = k[u];
          clear();
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float v[VEC];
          widen<In, VEC>(raw[u][e], v);
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[e][i] += v[i];
        }
      }
    }
  }
  const bool out_right = cur != none && cur == right;  // the last run goes on
  if (cur != none) {
    if (!inside)
      keep_head();
    else if (!out_right)
      put_rows(cur);
  }
  // the last group's lanes alone know whether the block's last run goes on
  const bool block_goes_on = __syncthreads_or(g == NG - 1 && out_right);
  auto goes_on = [&](int j) {  // group j's last run does not end with it
    return j + 1 < NG ? last[j] != none && last[j] == first[j + 1] : block_goes_on;
  };
  auto one_run = [&](int j) { return first[j] == last[j] && goes_on(j); };
  if (inside && out_right) {
    // a run that begins in this group: its parts to the right
    bool open = true;
    for (int j = g + 1; j < NG && open; ++j) {
      add_head(j);
      open = one_run(j);
    }
    if (open)
      put_part(part + a.Dp);
    else
      put_rows(cur);
  }
  if (g == 0 && n > 0 && first[0] != none && first[0] == left) {
    // the run that came in from the block before
    clear();
    add_head(0);
    for (int j = 0; j + 1 < NG && one_run(j); ++j) add_head(j + 1);
    put_part(part);
  }
}

// JOIN: the join kernel follows, and may be scheduled early (it waits before it
// reads anything; what else may follow is not known to). Blocks of an SM: four of bf16
// rows by 128 bits (16383 x 1000 36.8 us with three, 36.0 so, 36 to 56 bytes spilt a
// thread), three of the others (32768 x 64 f32 49.6 us, 51.1 with four). That rule
// was fitted to rows of 128-bit accesses: f32 pairs spill 88 to 148 bytes at its 80
// registers, and two blocks of them have not been measured.
template <class In, int VEC, int G, int E, bool JOIN>
__global__ void __launch_bounds__(kSumThreads, sizeof(In) == 2 && VEC > 2 ? 4 : 3)
    sum_kernel(const SumArgs a) {
  __shared__ SumSmem<VEC, G, E> sm;
  if constexpr (JOIN) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the sort (and the zeros) are done
  const int block = blockIdx.x / a.windows;
  const int64_t lo = static_cast<int64_t>(block) * a.per_block;
  sum_block<In, VEC, G, E>(a, sm, a.sorted, lo, min(lo + a.per_block, static_cast<int64_t>(a.T)),
                        a.chunk, blockIdx.x % a.windows,
                        a.part + static_cast<int64_t>(block) * 2 * a.Dp);
}

// The runs that begin in a block of chunks and go on past its end: their parts,
// added by eight warps in turn, for a window of columns. A join block for each
// block of chunks: most end after one look at the keys around the border.
// (Measured against 16 warps that look at as many borders and share long runs:
// 3.9 against 8.4 us at 256 blocks with several runs of 20, 12.9 against 12.4
// us with one of 460 blocks.)
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 128;  // columns of a join block: four a lane

// s += the parts of blocks from, from + step, .. to (slot 1 of block `start`, where
// the run begins, slot 0 of the others), eight loads in flight.
__device__ __forceinline__ void add_parts(const SumArgs& a, int start, int from, int to, int step,
                                          int c, float4& s) {
  for (int m0 = from; m0 <= to; m0 += 8 * step) {
    float4 p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int m = m0 + u * step;
      p[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m <= to)
        p[u] = *reinterpret_cast<const float4*>(
            a.part + (static_cast<int64_t>(m) * 2 + (m == start ? 1 : 0)) * a.Dp + c);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) s.x += p[u].x, s.y += p[u].y, s.z += p[u].z, s.w += p[u].w;
  }
}

__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const SumArgs a) {
  __shared__ float4 sums[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x;
  const int c = blockIdx.y * kJoinCols + lane * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are done
  const uint32_t none = a.rows;
  const int64_t begin = static_cast<int64_t>(i) * a.per_block, end = begin + a.per_block;
  // the first key of a block of chunks; `none` past the last
  auto first_key = [&](int m) {
    return m < a.nblocks ? a.sorted[static_cast<int64_t>(m) * a.per_block].x : none;
  };
  const uint32_t key = a.sorted[end - 1].x, next = first_key(i + 1);
  const uint32_t before = begin > 0 ? a.sorted[begin - 1].x : none;
  uint32_t reached = first_key(i + 2 + threadIdx.x);
  if (key == none || next != key || before == key) return;
  // the last block that the run reaches: those whose first key is the run's
  // follow each other
  int to = i + 1;
  for (int m0 = i + 2;; m0 += kJoinWarps * 32) {
    const int n = __syncthreads_count(reached == key);
    to += n;
    if (n < kJoinWarps * 32) break;
    reached = first_key(m0 + kJoinWarps * 32 + threadIdx.x);
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < a.Dp) add_parts(a, i, i + warp, to, kJoinWarps, c, s);
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
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

// Few tokens: all of the gradient in one launch, and no scratch. Every block
// ranks the tokens by counting the smaller keys (T^2 comparisons, kSmallTokens
// bounds them to about 2 us of a block) and takes a stretch of the sorted tokens
// that begins and ends with whole runs, for one window of columns; the zeros of
// the rows that no token names are shared out over all blocks, by a bitmap of
// the named rows in a block's share, in stores as wide as the rows allow (337 tokens
// of 9 bf16 into 286356 rows: 23 us with a block for each 32 KB, 15 with one for each
// eight stores a thread).

constexpr int kSmallTokens = 512;
constexpr int64_t kSmallZeros = 16 << 20;  // bytes of the gradient, at most
constexpr int kMapWords = 256;             // of the bitmap: rows / 32 at a time

struct SmallArgs {
  SumArgs sum;  // T, rows, ...: `sorted` and `part` are not used
  const int32_t* ids;
  int pad;
  FillArgs fill;
  int parts;  // of the tokens
  int32_t* status;
};

// Block `part` of `parts`: its share of the rows, without those in keys[0, T).
__device__ void fill_unnamed(const FillArgs& f, const uint32_t* keys, int T, int part, int parts,
                             uint32_t* map) {
  const int64_t begin = f.rows * part / parts, end = f.rows * (part + 1) / parts;
  const uint32_t per_row = static_cast<uint32_t>(f.row_bytes) / f.unit;
  for (int64_t r0 = begin; r0 < end; r0 += kMapWords * 32) {
    const int n = static_cast<int>(min(end - r0, static_cast<int64_t>(kMapWords * 32)));
    __syncthreads();
    for (int i = threadIdx.x; i < kMapWords; i += kSumThreads) map[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < T; i += kSumThreads) {
      const int64_t r = static_cast<int64_t>(keys[i]) - r0;
      if (r >= 0 && r < n) atomicOr(&map[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    const int64_t units = static_cast<int64_t>(n) * per_row;
    for (int64_t u = threadIdx.x; u < units; u += kSumThreads) {
      const uint32_t r = static_cast<uint32_t>(static_cast<uint32_t>(u) / per_row);
      if (map[r / 32] & (1u << (r % 32))) continue;
      put_zeros(f.out + (r0 + r) * f.pitch + (u - static_cast<int64_t>(r) * per_row) * f.unit,
                f.unit);
    }
  }
}

template <class In, int VEC, int G, int E>
__global__ void __launch_bounds__(kSumThreads) small_kernel(const SmallArgs a) {
  __shared__ SumSmem<VEC, G, E> sm;
  __shared__ __align__(16) uint32_t keys[kSmallTokens];
  __shared__ uint2 sorted[kSmallTokens];
  __shared__ uint32_t map[kMapWords];
  __shared__ int lo, hi;
  const int tid = threadIdx.x, T = a.sum.T;
  const uint32_t none = a.sum.rows;
  for (int i = tid; i < kSmallTokens; i += kSumThreads) {
    uint32_t key = 0xffffffffu;  // past the tokens: larger than any key
    if (i < T) {
      const int r = __ldg(a.ids + i);
      const bool in = static_cast<unsigned>(r) < none;
      if (!in && a.status != nullptr && blockIdx.x == 0)
        atomicOr(a.status, DLRM_FLAG_INDEX_OOB);
      key = (in && r != a.pad) ? r : none;
    }
    keys[i] = key;
  }
  const int part = blockIdx.x / a.sum.windows;
  if (tid == 0) lo = hi = T;
  __syncthreads();
  if (part < a.parts) {
    for (int i = tid; i < T; i += kSumThreads) {
      const uint32_t key = keys[i];
      int place = 0;
      for (int j = 0; j < T; j += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(&keys[j]);
        // equal keys: the earlier token first
        place += (k.x < key || (k.x == key && j < i)) + (k.y < key || (k.y == key && j + 1 < i)) +
                 (k.z < key || (k.z == key && j + 2 < i)) + (k.w < key || (k.w == key && j + 3 < i));
      }
      sorted[place] = make_uint2(key, static_cast<uint32_t>(i));
    }
    __syncthreads();
    // the part's first and last token, moved on to the next run's beginning
    const int from = static_cast<int>(static_cast<int64_t>(T) * part / a.parts);
    const int to = static_cast<int>(static_cast<int64_t>(T) * (part + 1) / a.parts);
    for (int i = tid; i < T; i += kSumThreads)
      if (i == 0 || sorted[i].x != sorted[i - 1].x) {
        if (i >= from) atomicMin(&lo, i);
        if (i >= to) atomicMin(&hi, i);
      }
    __syncthreads();
    constexpr int kGroups = SumSmem<VEC, G, E>::kGroups;
    const int per = (hi - lo + kGroups - 1) / kGroups;
    const int chunk = (per + kSumInFlight - 1) / kSumInFlight * kSumInFlight;
    if (hi > lo)
      sum_block<In, VEC, G, E>(a.sum, sm, sorted, lo, hi, chunk, blockIdx.x % a.sum.windows,
                               nullptr);
  }
  if (a.fill.out != nullptr)
    fill_unnamed(a.fill, keys, T, blockIdx.x, gridDim.x, map);
}

// The sums, then the runs that cross blocks. Launched kernels are added to n.
struct SumLaunch {
  SumArgs a;
  int n;
  cudaStream_t stream;
  template <class In, int VEC, int G, int E>
  cudaError_t run() {
    constexpr int kWindow = G * E * VEC;
    a.windows = (a.D + kWindow - 1) / kWindow;
    a.per_block = a.chunk * (kSumThreads / G);
    a.nblocks = static_cast<int>((static_cast<int64_t>(a.T) + a.per_block - 1) / a.per_block);
    const int64_t blocks = static_cast<int64_t>(a.nblocks) * a.windows;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e =
        launch(a.nblocks > 1 ? &sum_kernel<In, VEC, G, E, true> : &sum_kernel<In, VEC, G, E, false>,
               dim3(static_cast<unsigned>(blocks)), kSumThreads, 0, true, stream, a);
    if (e != cudaSuccess) return e;
    ++n;
    if (a.nblocks > 1) {
      const dim3 grid(a.nblocks - 1, (a.D + kJoinCols - 1) / kJoinCols);
      e = launch(&join_kernel, grid, kJoinWarps * 32, 0, true, stream, a);
      ++n;
    }
    return e;
  }
};

// All of it in one launch, for few tokens.
struct SmallLaunch {
  SmallArgs a;
  cudaStream_t stream;
  template <class In, int VEC, int G, int E>
  cudaError_t run() {
    constexpr int kWindow = G * E * VEC;
    a.sum.windows = (a.sum.D + kWindow - 1) / kWindow;
    constexpr int per_block = kSumThreads / G * kSumInFlight;  // tokens in flight
    a.parts = (a.sum.T + per_block - 1) / per_block;
    // blocks: for the sums, and for the zeros, eight stores a thread
    int64_t blocks = static_cast<int64_t>(a.parts) * a.sum.windows;
    if (a.fill.out != nullptr)
      blocks = std::max(blocks, std::min<int64_t>(
                                    kSms * 8, a.fill.rows * a.fill.row_bytes /
                                                  (8 * kSumThreads * a.fill.unit)));
    return launch(&small_kernel<In, VEC, G, E>, dim3(static_cast<unsigned>(blocks)), kSumThreads, 0,
                  false, stream, a);
  }
};

// Sizes of a gradient's scratch, and where its parts lie.
struct GradPlan {
  int sort_blocks, per, items, passes, bits;
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
  // tiles that give about two blocks an SM while one tile a block will do (4608
  // pairs: up to 1.36 M tokens), whole tiles of 8192 pairs a block beyond
  const int64_t share = (T + kSortMaxBlocks - 1) / kSortMaxBlocks;
  p.items = share <= kSortThreads * 4   ? 4
            : share <= kSortThreads * 6 ? 6
            : share <= kSortThreads * 9 ? 9
                                        : kSortItems;
  const int64_t tile = kSortThreads * p.items;
  const int64_t per = std::max<int64_t>(1, (share + tile - 1) / tile) * tile;
  p.per = static_cast<int>(per);
  p.sort_blocks = static_cast<int>((T + per - 1) / per);
  // a group's tokens: as few as are in flight at once while that fills the
  // GPU's threads, more when there are more; by T and D alone. (16383 x 1000
  // takes 36 us with 8 tokens, 34 with 16, 36 with 24; 32768 x 64 51.3,
  // 51.7 and 53.3.)
  const int64_t even = T * D / (int64_t{kSms} * 2048 * 4) / kSumInFlight + 1;
  p.chunk = static_cast<int>(std::min<int64_t>(64, even * kSumInFlight));
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
  // the one-launch form (for f32 and accumulating or not, so that the size alone
  // decides) keeps everything in shared memory
  p.bytes = T <= kSmallTokens && rows * D <= kSmallZeros / 4 ? 0 : at;
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
  const int vec = common_vec(table, ldw, es, out, ldo, os, D);
  cudaError_t e;
  if (out_dtype == DLRM_TABLE_F32) {
    LookupLaunch<float> f = {a, s};
    e = by_type(table_dtype, a.D, vec, f);
  } else {
    LookupLaunch<__nv_bfloat16> f = {a, s};
    e = by_type(table_dtype, a.D, vec, f);
  }
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
  if (p.bytes > 0 && scratch == nullptr) return DLRM_ERR_NULL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = clear_status(status_dev, s);
  if (rc != DLRM_OK) return rc;
  const int sms = sm_count_current();
  if (sms == 0) return DLRM_ERR_CUDA;
  FillArgs fill = {};
  if (!accumulate) {
    fill.out = static_cast<char*>(out);
    fill.rows = rows;
    fill.row_bytes = D * os;
    fill.pitch = ldo * os;
    fill.unit = os;
    for (int u : {4, 8, 16})
      if (((reinterpret_cast<intptr_t>(fill.out) | fill.row_bytes | fill.pitch) & (u - 1)) == 0)
        fill.unit = u;
  }
  if (T == 0) {
    if (accumulate) return DLRM_OK;
    const cudaError_t e = run_fill<false>(fill, sms, s);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch();
    return DLRM_OK;
  }

  SumArgs a = {};
  a.grad = grad;
  a.ldg = ldg;
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
  const int vec = common_vec(grad, ldg, es, out, ldo, os, D);
  cudaError_t e;
  if (T <= kSmallTokens && (accumulate || rows * D * os <= kSmallZeros)) {
    SmallLaunch f = {};
    f.a.sum = a;
    f.a.ids = ids;
    f.a.pad = static_cast<int>(padding_idx);
    f.a.fill = fill;
    f.a.status = status_dev;
    f.stream = s;
    if ((e = by_type(grad_dtype, a.D, vec, f)) != cudaSuccess) return cuda_fail(e);
    note_launch();
    return DLRM_OK;
  }

  char* mem = static_cast<char*>(scratch);
  SortArgs sa = {};
  sa.ids = ids;
  sa.counts = reinterpret_cast<uint32_t*>(mem + p.counts);
  sa.T = static_cast<int>(T);
  sa.rows = static_cast<int>(rows);
  sa.pad = static_cast<int>(padding_idx);
  sa.bits = p.bits;
  sa.passes = p.passes;
  sa.per = p.per;
  sa.blocks = p.sort_blocks;
  sa.fill = fill;
  sa.status = status_dev;
  uint2* const pairs[2] = {reinterpret_cast<uint2*>(mem + p.pairs[0]),
                           reinterpret_cast<uint2*>(mem + p.pairs[1])};
  sa.out = pairs[0];
  int n = 0;
  if (T <= kClusterSort) {
    const int64_t items = (T + kClusterSize * kClusterThreads - 1) / (kClusterSize * kClusterThreads);
    e = items <= 1   ? run_cluster_sort<1>(sa, sms, n, s)
        : items <= 2 ? run_cluster_sort<2>(sa, sms, n, s)
        : items <= 4 ? run_cluster_sort<4>(sa, sms, n, s)
                     : run_cluster_sort<8>(sa, sms, n, s);
  } else {
    if (fill.out != nullptr && fill.apart()) {
      if ((e = run_fill<false>(fill, sms, s)) != cudaSuccess) return cuda_fail(e);
      sa.fill.out = nullptr;
      ++n;
    }
    e = p.items == 4   ? run_grid_sort<4>(sa, pairs, s)
        : p.items == 6 ? run_grid_sort<6>(sa, pairs, s)
        : p.items == 9 ? run_grid_sort<9>(sa, pairs, s)
                       : run_grid_sort<kSortItems>(sa, pairs, s);
    n += 2 * p.passes;
  }
  if (e != cudaSuccess) return cuda_fail(e);
  a.sorted = sa.out;
  a.part = reinterpret_cast<float*>(mem + p.part);
  SumLaunch f = {a, n, s};
  if ((e = by_type(grad_dtype, a.D, vec, f)) != cudaSuccess) return cuda_fail(e);
  note_launch(f.n);
  return DLRM_OK;
}

}  // extern "C"
