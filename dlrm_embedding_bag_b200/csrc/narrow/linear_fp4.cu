// The layer on 4-bit floating point (declared in dlrm_fp4.h):
// y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]).
//
// tcgen05.mma.kind::mxf4.block_scale: products of e2m1 codes times both blocks'
// powers of two, K = 64 an instruction, f32 sums in TMEM.
//
// Fourteen warps a CTA: one thread streams 128-byte K blocks (256 elements) of both
// operands and their scale tiles into a shared-memory ring with TMA loads; four warps
// carry a stage's scales from there into TMEM, up to four stages ahead; one thread
// issues a stage's four products; eight warps drain a finished accumulator while the
// next tile's products fill the other. (tcgen05.cp brings scales to TMEM as well, but in
// the tensor cores' own queue: a stage's six copies held up its products by 0.15 of 0.63
// us, 8192^3 284 us where this took 240.)
//
// Forms:
//   - CTAs of 128 channels x 64 or 128 tokens: the weights take the M side, so an
//     accumulator lane is a channel, few tokens make a narrow tile, and the 32 lanes of a
//     warp store 32 neighbouring channels of a token at any pitch. Few tiles: a
//     cluster of S CTAs shares one tile, each summing a stretch of K, and the f32 parts
//     meet through distributed shared memory in the order of the ranks.
//   - CTA pairs (cta_group::2) of 256 x 256. Where rows of y are whole 16 bytes the
//     tokens take the M side: a lane then has neighbouring channels of a token, lays
//     them out in shared memory, and the copy engine writes whole lines. Two accumulators of 256 columns and
//     the scales do not fit TMEM's 512, so the accumulators share 128 columns: those
//     are drained first, and the next tile's products wait for that.
//   - one token: CUDA cores (below).
// Every wait is bounded; one that runs out sets DLRM_FLAG_TIMEOUT in the
// optional status word, and the CTA still lets its loads land, frees its tensor
// memory and exits.
#include <algorithm>
#include <atomic>
#include <climits>

#include "fp4_common.cuh"
#include "fp4_forms.h"
#include "ring_landing.h"
#include "sectors.cuh"
#include "tcgen05_common.cuh"
#include "tokens/common.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBM = 128;            // channels of a CTA's tile
constexpr int kBK = 128;            // bytes of K per stage: one 128-byte swizzle row
constexpr int kCols = 2 * kBK;      // elements of K per stage
constexpr int kStageTiles = kCols / 128;  // scale tiles along K per stage
constexpr int kEpiWarps = 8;
constexpr int kScaleWarp = 2 + kEpiWarps;  // the first of the four that carry scales
constexpr int kThreads = 32 * (kScaleWarp + 4);
constexpr long long kWaitLimit = 200000000LL;  // clock cycles, about 0.1 s
// What a wait for a whole tile's products may take besides, for each of its stages (which
// take 300 to 800 cycles): 2^22 stages of a K of 2^30 are more than the limit above.
constexpr long long kStageLimit = 10000;
constexpr int kMaxDevices = 64;                // devices whose launch set-up is cached

constexpr int kBand = 8;  // tiles of b that are walked together
// The operand on the M side is a (the weights, or with TOKENS_M the tokens), the other b.
struct LinArgs {
  const float* bias;
  void* y;
  int64_t ldy;
  int na, nb, K;                 // rows of a and of b
  int nkb;                       // K blocks
  int tiles_a, tiles_b, tiles;
  Divisor by_band;               // a band's tiles
  int act, y_bf16;
  int32_t* status;
};

struct alignas(64) LinMaps {
  CUtensorMap a, b, sa, sb, y;  // y: with TOKENS_M
};

// Shared memory and TMEM of a form. BN rows of b a tile; a pair's CTA loads half of them,
// but the scales of all, which each CTA's tensor cores read from its own TMEM.
// OUT: with room for each epilogue warp's part of y on its way out.
constexpr int kOutBytes = 4096;  // 32 rows of 128 bytes
template <int BN, bool PAIR, bool OUT>
struct Ring {
  static constexpr int kBTiles = BN > 128 ? BN / 128 : 1;  // row tiles of b's scales
  static constexpr int kA = kBM * kBK;
  static constexpr int kB = (PAIR ? BN / 2 : BN) * kBK;
  static constexpr int kSA = kStageTiles * kFp4Tile;
  static constexpr int kSB = kBTiles * kStageTiles * kFp4Tile;
  static constexpr int kStage = kA + kB + kSA + kSB;
  // as many stages as fit in about 180 or 200 KB, at most 8
  static constexpr int kRoom = (OUT ? 180 : 200) * 1024;
  static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
  static constexpr int kOut = kStages * kStage;
  static constexpr int kBias = kOut + kEpiWarps * kOutBytes;  // a slice of it for each warp
  static constexpr int kBars = OUT ? kBias + kEpiWarps * (BN / 2) * 4 : kOut;
  // stages whose scales are in TMEM at a time
  static constexpr int kCarried = 4;
  static constexpr int kBarriers = 3 * kStages + kCarried + 6;
  static constexpr int kTotal = kBars + kBarriers * 8 + 8 + 1024;  // + alignment
  static_assert(kStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
  static_assert(kStages >= kCarried, "a column set is free when its stage's place is");
  static_assert(kTotal <= 227 * 1024, "shared memory of one CTA");
  // TMEM columns: the second accumulator, the scales, and what both accumulators have
  // of each other
  static constexpr int kLap = BN > 128 ? 128 : 0;
  static constexpr uint32_t kAcc1 = BN - kLap;
  static constexpr uint32_t kScales = kAcc1 + BN;
  static constexpr uint32_t kScaleCols = 4 * kStageTiles * (1 + kBTiles);
  static constexpr uint32_t kNeeded = kScales + kCarried * kScaleCols;
  static constexpr uint32_t kTmem = kNeeded <= 256 ? 256 : 512;
  static_assert(kNeeded <= 512, "tensor memory of one SM");
};

// Instruction descriptor of tcgen05.mma.kind::mxf4.block_scale with e2m1 A and B, both
// K-major, UE8M0 scales, dense, K = 64, shape M x N: B's scale bytes (bits 4-5), A and B
// formats E2M1 (7-9 = 1, 10-12 = 1), N >> 3 (17-22), scales UE8M0 (23 = 1), M >> 4 (24-28),
// A's scale bytes (29-30). The scale bytes of a product are a pair of a column's
// four: 0 for the first, 2 for the second.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, uint32_t pair) {
  return (pair << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) | (pair << 29);
}

// D[tmem] (+)= A[smem] * B[smem]^T for one K = 64 step of 4-bit elements with scales in TMEM.
template <int CG>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t sa, uint32_t sb,
                                           uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
        "[%6], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
        "[%6], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb)
        : "memory");
}

// The same one of a whole warp's lanes at every call.
__device__ __forceinline__ bool elected() {
  uint32_t mine;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(mine));
  return mine != 0;
}

// N 32-bit columns of the warp's 32 TMEM lanes, from each lane's registers.
__device__ __forceinline__ void tmem_st_8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                   taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The box of a 3-D tensor map at (x, y, z), as tma_load_2d.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

__device__ __forceinline__ float4 load_cluster_v4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == DLRM_ACT_RELU) return x < 0.f ? 0.f : x;  // NaN stays NaN
  if constexpr (ACT == DLRM_ACT_SIGMOID) return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x)));
  return x;
}

template <int ACT, class Out>
__device__ __forceinline__ void put_at(Out* p, float sum, float bias) {
  const float v = activate<ACT>(__fadd_rn(sum, bias));
  if constexpr (sizeof(Out) == 4)
    *p = v;
  else
    *p = __float2bfloat16_rn(v);
}

// b's rows b0 .. b0 + 31 (tokens) of a lane's row of a (a channel), from the registers v.
template <int ACT, class Out>
__device__ __forceinline__ void put_tokens(const LinArgs& a, int row, float bias, int b0,
                                           const float* v) {
  if (row >= a.na) return;
  Out* p = static_cast<Out*>(a.y) + static_cast<int64_t>(b0) * a.ldy + row;
  const int left = a.nb - b0;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float lo = activate<ACT>(__fadd_rn(v[i], bias)), hi = activate<ACT>(__fadd_rn(v[i + 1], bias));
    if constexpr (sizeof(Out) == 4) {
      if (i < left) p[0] = lo;
      if (i + 1 < left) p[a.ldy] = hi;
    } else {
      const uint32_t both = bf16_pair(lo, hi);
      uint16_t* at = reinterpret_cast<uint16_t*>(p);
      if (i < left) at[0] = static_cast<uint16_t>(both);
      if (i + 1 < left) at[a.ldy] = static_cast<uint16_t>(both >> 16);
    }
    p += 2 * a.ldy;
  }
}

// b's rows b0 .. b0 + 63 (channels) of 32 rows of a from row0 on (tokens), one a lane: laid
// out in shared memory as the map's 128-byte swizzle has it, and from there to y by the
// copy engine, which leaves out what is past y's end. Rows of y are whole 16 bytes. bias: of
// these channels, in shared memory.
template <int ACT, class Out>
__device__ __forceinline__ void put_channels(const LinArgs& a, const CUtensorMap* y, uint8_t* out,
                                             int row0, int b0, int lane, const float* bias,
                                             float* v) {
  constexpr int kPiece = 16 / sizeof(Out), kAtOnce = 8 * kPiece;  // columns of 16 and 128 bytes
  // all of the bias before anything is stored, which a load could not pass
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(bias + i);
    v[i] = activate<ACT>(__fadd_rn(v[i], f.x));
    v[i + 1] = activate<ACT>(__fadd_rn(v[i + 1], f.y));
    v[i + 2] = activate<ACT>(__fadd_rn(v[i + 2], f.z));
    v[i + 3] = activate<ACT>(__fadd_rn(v[i + 3], f.w));
  }
#pragma unroll
  for (int c = 0; c < 64; c += kAtOnce) {
    if (lane == 0) bulk_wait_read_all();  // the last ones have been read
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p)
      store_16_bytes(reinterpret_cast<Out*>(out + lane * 128 + ((p ^ (lane & 7)) << 4)),
                     v + c + p * kPiece);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row0 < a.na && b0 + c < a.nb) {
      tma_store_2d(y, out, b0 + c, row0);
      bulk_commit();
    }
  }
}

// Calls f with the activation and the output type as types.
template <class Args, class F>
__device__ __forceinline__ void by_kind(const Args& a, F f) {
  if (a.y_bf16) {
    if (a.act == DLRM_ACT_RELU)
      f.template run<DLRM_ACT_RELU, __nv_bfloat16>();
    else if (a.act == DLRM_ACT_SIGMOID)
      f.template run<DLRM_ACT_SIGMOID, __nv_bfloat16>();
    else
      f.template run<DLRM_ACT_NONE, __nv_bfloat16>();
  } else {
    if (a.act == DLRM_ACT_RELU)
      f.template run<DLRM_ACT_RELU, float>();
    else if (a.act == DLRM_ACT_SIGMOID)
      f.template run<DLRM_ACT_SIGMOID, float>();
    else
      f.template run<DLRM_ACT_NONE, float>();
  }
}

struct PutTokens {
  const LinArgs& a;
  int row, b0;
  float bias;
  const float* v;
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    put_tokens<ACT, Out>(a, row, bias, b0, v);
  }
};
struct PutChannels {
  const LinArgs& a;
  const CUtensorMap* y;
  uint8_t* out;
  int row0, b0, lane;
  const float* bias;
  float* v;
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    put_channels<ACT, Out>(a, y, out, row0, b0, lane, bias, v);
  }
};

// The cluster's parts of a tile, kept as [column][channel] f32 at the start of each CTA's
// ring, summed in the order of its S CTAs for columns [c0, c1): a column's 128 channels a
// warp, four a lane, the loads of eight parts in flight.
template <int S>
struct JoinCall {
  const LinArgs& a;
  int a0, b0, c0, c1, ew, lane;
  uint32_t smem;
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    constexpr int kAtOnce = 8 / S;  // columns
    const int n = a0 + lane * 4;
    float bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = a.bias != nullptr && n + e < a.na ? a.bias[n + e] : 0.f;
    for (int cb = c0 + ew * kAtOnce; cb < c1; cb += kEpiWarps * kAtOnce) {
      float4 v[kAtOnce][S];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
        for (int k = 0; k < S; ++k) {
          v[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (cb + i < c1 && b0 + cb + i < a.nb)
            v[i][k] = load_cluster_v4(map_to_cta(smem + ((cb + i) * kBM + lane * 4) * 4, k));
        }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (cb + i >= c1 || b0 + cb + i >= a.nb) break;
        float4 t = v[i][0];
#pragma unroll
        for (int k = 1; k < S; ++k)
          t.x += v[i][k].x, t.y += v[i][k].y, t.z += v[i][k].z, t.w += v[i][k].w;
        const float sums[4] = {t.x, t.y, t.z, t.w};
        Out* p = static_cast<Out*>(a.y) + static_cast<int64_t>(b0 + cb + i) * a.ldy + n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.na) put_at<ACT>(p + e, sums[e], bias[e]);
      }
    }
  }
};

// Tile t -> (tile of a, tile of b): bands of kBand tiles of b, so that the CTAs at work at one
// time read few different rows of either operand.
__device__ __forceinline__ void tile_at(const LinArgs& a, int t, int& ta, int& tb) {
  const int band = static_cast<int>(a.by_band.of(t)), in = t - band * (kBand * a.tiles_a);
  const int height = min(kBand, a.tiles_b - band * kBand);
  if (height == kBand) {
    tb = band * kBand + in % kBand;
    ta = in / kBand;
  } else {
    tb = band * kBand + in % height;
    ta = in / height;
  }
}

// S > 1: the S CTAs of a cluster share one tile (and there is one tile a cluster).
template <int BN, bool PAIR, int S, bool TOKENS_M>
__global__ void __launch_bounds__(kThreads, 1)
    linear_fp4_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs args) {
  constexpr bool SPLIT = S > 1;
  static_assert(!(PAIR && SPLIT), "a pair shares a tile's rows of a, not its K");
  static_assert(!(TOKENS_M && SPLIT), "parts are joined channel by channel");
  using R = Ring<BN, PAIR, TOKENS_M>;
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int kUnitA = CG * kBM;                          // rows of a in a unit's tile
  constexpr int kWarpCols = BN / 2;                         // columns an epilogue warp drains
  constexpr int kAtOnce = kWarpCols < 64 ? kWarpCols : 64;  // of them at a time
  static_assert(kAtOnce % 32 == 0, "whole TMEM loads");
  static_assert(R::kLap == 0 || (R::kLap == 2 * kAtOnce && BN == 4 * kAtOnce),
                "the shared columns are a step of all warps");
  static_assert(!TOKENS_M || kAtOnce == 64, "whole lines of y");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + R::kBars);  // codes are there
  uint64_t* scales = full + R::kStages;                           // this CTA's scale tiles are
  uint64_t* empty = scales + R::kStages;
  uint64_t* carried = empty + R::kStages;                         // scales are in TMEM
  uint64_t* acc_full = carried + R::kCarried;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_done = acc_empty + 2;
  uint64_t* lap_empty = mma_done + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(lap_empty + 1);
  uint32_t* other_steps = tslot + 1;  // of a pair's second producer, told at its end
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = (PAIR || SPLIT) ? cluster_ctarank() : 0u;
  const int unit0 = (PAIR || SPLIT) ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int unit_step =
      (PAIR || SPLIT) ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  // this CTA's stretch of K blocks
  const int kb_begin = SPLIT ? static_cast<int>(static_cast<int64_t>(args.nkb) * rank / S) : 0;
  const int kb_end = SPLIT ? static_cast<int>(static_cast<int64_t>(args.nkb) * (rank + 1) / S) : args.nkb;

  if (warp == 1) {
    tmem_alloc<CG>(tslot, R::kTmem);
    tmem_relinquish<CG>();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < R::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&scales[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < R::kCarried; ++s) mbar_init(&carried[s], CG * 4);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CG * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    mbar_init(lap_empty, CG * kEpiWarps);
    mbar_init_fence();
    if constexpr (PAIR) *other_steps = ~0u;
  }
  tc_fence_before_sync();
  if constexpr (PAIR)
    cluster_sync();  // both CTAs' barriers exist before either signals the other's
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tslot;
  // Everything below may come from the kernel before, which may still be at work, so every
  // role waits for its end. The loads behind the wait are ordinary ones: those of the
  // read-only path may be moved in front of it.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool timed_out = false;
  // a whole warp's arrival, for reads or writes of tensor memory that the issuer of the
  // products (a pair's first CTA) waits for
  auto arrive = [&](uint64_t* bar) {
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      if constexpr (PAIR)
        mbar_arrive_remote(map_to_cta(smem_u32(bar), 0));
      else
        mbar_arrive(bar);
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      int g = 0;
      for (int t = unit0; t < args.tiles && !timed_out; t += unit_step) {
        int ta, tb;
        tile_at(args, t, ta, tb);
        const int a0 = ta * kUnitA + (PAIR ? static_cast<int>(rank) * kBM : 0);
        const int b0 = tb * BN + (PAIR ? static_cast<int>(rank) * (BN / 2) : 0);
        for (int kb = kb_begin; kb < kb_end; ++kb, ++g) {
          const int s = g % R::kStages;
          if (g >= R::kStages &&
              !mbar_wait_bounded(&empty[s], ((g / R::kStages) - 1) & 1, kWaitLimit)) {
            timed_out = true;
            break;
          }
          uint8_t* sa = smem + s * R::kStage;
          uint8_t* sb = sa + R::kA;
          uint8_t* ssa = sb + R::kB;
          uint8_t* ssb = ssa + R::kSA;
          // a CTA's scale tiles are counted on its own barrier
          mbar_arrive_expect_tx(&scales[s], R::kSA + R::kSB);
          tma_load_3d(ssa, &maps.sa, &scales[s], 0, kb * kStageTiles, a0 / 128);
          tma_load_3d(ssb, &maps.sb, &scales[s], 0, kb * kStageTiles, tb * BN / 128);
          if constexpr (PAIR) {
            // both CTAs' codes are counted on the issuer's barrier, which only its
            // producer arms
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (R::kA + R::kB));
            const uint32_t fb = map_to_cta(smem_u32(&full[s]), 0);
            tma_load_2d_pair(sa, &maps.a, fb, kb * kBK, a0);
            tma_load_2d_pair(sb, &maps.b, fb, kb * kBK, b0);
          } else {
            mbar_arrive_expect_tx(&full[s], R::kA + R::kB);
            tma_load_2d(sa, &maps.a, &full[s], kb * kBK, a0);
            tma_load_2d(sb, &maps.b, &full[s], kb * kBK, b0);
          }
        }
      }
      // no load is in flight once this CTA leaves, whoever gave up
      land_loads<R::kStages, false>(
          true, timed_out, g,
          [&](int s, uint32_t parity) { (void)mbar_wait_bounded(&scales[s], parity, kWaitLimit); },
          [](int) {}, [](int) {}, [] { return -1; });
      land_loads<R::kStages, PAIR>(
          !PAIR || rank == 0, timed_out, g,
          [&](int s, uint32_t parity) { (void)mbar_wait_bounded(&full[s], parity, kWaitLimit); },
          [&](int s) { mbar_arrive_expect_tx(&full[s], R::kA + R::kB); },
          [&](int steps) { tell_steps(other_steps, steps); },
          [&] { return told_steps(other_steps, (R::kStages + 2) * kWaitLimit); });
    }
  } else if (warp == 1) {
    // The whole warp walks the stages and one elected lane issues: what the products' operands are
    // made of is then the same for the warp and stays in its uniform registers (by one
    // lane alone a stage of a pair took 911 cycles, so 680).
    if (!PAIR || rank == 0) {
      const uint64_t a_desc = sdesc_k_sw128(smem_u32(smem));
      const uint64_t b_desc = sdesc_k_sw128(smem_u32(smem) + R::kA);
      int j = 0, s = 0, c = 0;
      uint32_t s_turn = 0, c_turn = 0;  // parities of the ring's and the column sets' turns
      for (int t = unit0; t < args.tiles && !timed_out; t += unit_step, ++j) {
        const int b = j & 1;
        bool ok = j < 2 || mbar_wait_bounded(&acc_empty[b], ((j >> 1) - 1) & 1, kWaitLimit);
        if (R::kLap != 0 && ok && j >= 1) ok = mbar_wait_bounded(lap_empty, (j - 1) & 1, kWaitLimit);
        if (!__all_sync(kFull, ok)) {
          timed_out = true;
          break;
        }
        const uint32_t acc = tmem + (b != 0 ? R::kAcc1 : 0u);
        // rows of b from the middle of a scale tile on: 32 rows of it are a column
        int ta, tb;
        tile_at(args, t, ta, tb);
        const uint32_t b_col = static_cast<uint32_t>(tb * BN % 128 / 32);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          if (!__all_sync(kFull, mbar_wait_bounded(&full[s], s_turn, kWaitLimit) &&
                                     mbar_wait_bounded(&carried[c], c_turn, kWaitLimit))) {
            timed_out = true;
            break;
          }
          tc_fence_after_sync();
          const uint64_t ad = a_desc + static_cast<uint32_t>(s * (R::kStage >> 4));
          const uint64_t bd = b_desc + static_cast<uint32_t>(s * (R::kStage >> 4));
          const uint32_t ca = tmem + R::kScales + static_cast<uint32_t>(c) * R::kScaleCols;
          const uint32_t cb = ca + 4 * kStageTiles + b_col;
          // products past K would add zeros
          const int steps = min(4, (args.K - kb * kCols + 63) / 64);
          if (elected()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < steps)
                tc_mma_fp4<CG>(acc, ad + 2 * k, bd + 2 * k, idesc_mxf4(kUnitA, BN, 2 * (k & 1)),
                               ca + 4 * (k >> 1), cb + 4 * (k >> 1) * R::kBTiles,
                               (kb > kb_begin || k > 0) ? 1u : 0u);
            if constexpr (PAIR)
              tc_commit_pair_both(&empty[s]);
            else
              tc_commit<CG>(&empty[s]);
          }
          __syncwarp();
          if (++s == R::kStages) s = 0, s_turn ^= 1;
          if (++c == R::kCarried) c = 0, c_turn ^= 1;
        }
        if (elected()) {
          if constexpr (PAIR)
            tc_commit_pair_both(&acc_full[b]);
          else
            tc_commit<CG>(&acc_full[b]);
        }
        __syncwarp();
      }
      // every MMA has completed before this CTA or its peer can leave
      if (elected()) tc_commit<CG>(mma_done);
      __syncwarp();
      if (!mbar_wait_bounded(mma_done, 0, kWaitLimit)) timed_out = true;
    }
  } else if (warp >= kScaleWarp) {
    // A stage's scale tiles: lane i of every warp takes the 16 bytes of rows i, i + 32, i +
    // 64 and i + 96, four columns of its TMEM lane. A column set is free once the products of
    // the stage that had it before are done, which is when its place in the ring is.
    const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int g = 0;
    for (int t = unit0; t < args.tiles && !timed_out; t += unit_step) {
      for (int kb = kb_begin; kb < kb_end; ++kb, ++g) {
        const int s = g % R::kStages, c = g % R::kCarried, before = g - R::kCarried;
        bool ok = mbar_wait_bounded(&scales[s], (g / R::kStages) & 1, kWaitLimit);
        if (ok && before >= 0)
          ok = mbar_wait_bounded(&empty[before % R::kStages], (before / R::kStages) & 1, kWaitLimit);
        if (!__all_sync(kFull, ok)) {
          timed_out = true;
          break;
        }
        tc_fence_after_sync();
        const uint8_t* tile = smem + s * R::kStage + R::kA + R::kB + lane * 16;
        const uint32_t to = tmem + quarter + R::kScales + static_cast<uint32_t>(c) * R::kScaleCols;
        uint32_t r[R::kScaleCols];
#pragma unroll
        for (int i = 0; i < kStageTiles * (1 + R::kBTiles); ++i) {
          // a's tiles along K, then b's: along K, of each its row tiles
          const int b = i - kStageTiles;
          const int at = i < kStageTiles ? i : kStageTiles + b % R::kBTiles * kStageTiles + b / R::kBTiles;
          const uint4 v = *reinterpret_cast<const uint4*>(tile + at * kFp4Tile);
          r[4 * i] = v.x, r[4 * i + 1] = v.y, r[4 * i + 2] = v.z, r[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < static_cast<int>(R::kScaleCols); i += 8) tmem_st_8(to + i, r + i);
        tmem_st_wait();
        arrive(&carried[c]);
      }
    }
  } else {
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    // TOKENS_M: a warp's bias of a tile, a few columns a lane, on its way since the tile before
    constexpr int kMine = kWarpCols / 32;
    float next[kMine] = {};
    auto fetch_bias = [&](int t) {
      if (!TOKENS_M || args.bias == nullptr || t >= args.tiles) return;
      int ta, tb;
      tile_at(args, t, ta, tb);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int c = 32 * i + lane;
        const int n = tb * BN + (c / kAtOnce * 2 + half) * kAtOnce + c % kAtOnce;
        next[i] = n < args.nb ? args.bias[n] : 0.f;
      }
    };
    fetch_bias(unit0);
    int j = 0;
    for (int t = unit0; t < args.tiles; t += unit_step, ++j) {
      const int b = j & 1;
      int ta, tb;
      tile_at(args, t, ta, tb);
      const int b0 = tb * BN;
      const int row = ta * kUnitA + (PAIR ? static_cast<int>(rank) * kBM : 0) + quarter * 32 + lane;
      float bias = 0.f;
      if (!SPLIT && !TOKENS_M && row < args.na && args.bias != nullptr) bias = args.bias[row];
      float* slice = reinterpret_cast<float*>(smem + R::kBias) + ew * kWarpCols;
      if constexpr (TOKENS_M) {
        __syncwarp();  // the slice's readers of the tile before are done
#pragma unroll
        for (int i = 0; i < kMine; ++i) slice[32 * i + lane] = next[i];
        __syncwarp();
        fetch_bias(t + unit_step);
      }
      if (!__all_sync(kFull, mbar_wait_bounded(&acc_full[b], (j >> 1) & 1,
                                               kWaitLimit + (kb_end - kb_begin) * kStageLimit))) {
        timed_out = true;
        break;
      }
      tc_fence_after_sync();
      const uint32_t tq = tmem + (b != 0 ? R::kAcc1 : 0u) + (static_cast<uint32_t>(quarter * 32) << 16);
      // A step is 64 columns a warp, those of the two halves of warps next to each other. The
      // columns that the next tile's accumulator has too come first: the upper ones of the
      // lower accumulator, the lower ones of the upper one.
      constexpr int kSteps = kWarpCols / kAtOnce;
      for (int i = 0; i < kSteps; ++i) {
        const int step = kSteps == 2 ? (i + 1 - b) & 1 : i;
        const int c = (2 * step + half) * kAtOnce;
        float v[kAtOnce];
#pragma unroll
        for (int h = 0; h < kAtOnce; h += 32)
          tmem_ld_32x32b_x32(tq + c + h, *reinterpret_cast<float(*)[32]>(v + h));
        if (R::kLap != 0 && i == 0) arrive(lap_empty);
        if (i == kSteps - 1) arrive(&acc_empty[b]);
        if constexpr (TOKENS_M) {
          by_kind(args, PutChannels{args, &maps.y, smem + R::kOut + ew * kOutBytes, row - lane,
                                    b0 + c, lane, slice + step * kAtOnce, v});
        } else {
#pragma unroll
          for (int h = 0; h < kAtOnce; h += 32) {
            if constexpr (SPLIT) {
              // all products are done: the ring is free for this CTA's part
              float* part = reinterpret_cast<float*>(smem);
#pragma unroll
              for (int e = 0; e < 32; ++e) part[(c + h + e) * kBM + quarter * 32 + lane] = v[h + e];
            } else if (b0 + c + h < args.nb) {
              by_kind(args, PutTokens{args, row, b0 + c + h, bias, v + h});
            }
          }
        }
        __syncwarp();  // the next load takes the whole warp
      }
    }
    if (TOKENS_M && lane == 0) bulk_wait_all();
  }
  if (timed_out && args.status != nullptr) atomicOr(args.status, DLRM_FLAG_TIMEOUT);
  if constexpr (SPLIT) {
    cluster_sync();  // every CTA's part is in its shared memory
    if (warp >= 2 && warp < kScaleWarp) {
      int ta, tb;
      tile_at(args, unit0, ta, tb);
      const int c0 = BN * static_cast<int>(rank) / S, c1 = BN * static_cast<int>(rank + 1) / S;
      by_kind(args, JoinCall<S>{args, ta * kBM, tb * BN, c0, c1, warp - 2, lane, smem_u32(smem)});
    }
  }
  tc_fence_before_sync();
  if constexpr (PAIR || SPLIT)
    cluster_sync();  // no CTA leaves while another may still use its memory
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc<CG>(tmem, R::kTmem);
}

// One token: R channels a warp, a lane for each block of 32 columns, U of them at a time.
// Codes become twice their values as 8-bit integers (a byte permutation looks four up in a
// register pair), four products an instruction; a block's sum is exact in int32 and scaled
// once. The token's codes are looked up once for the warp's channels. A trip over the row takes 32 U
// blocks, and its weights are on their way before the first of them is used; the next trip's are not.
// Bound by latency: 4096 x 4096 takes 4.9 us with weights in L2 and 5.7 with weights from HBM, 1.4 by
// its bytes. It is two trips by 1.7 CTAs an SM; 0.31 instructions a scheduler and cycle of 1.7
// warps, which wait for loads most, and the pipe of the permutations at 30 %.
constexpr int kOneThreads = 128;

struct OneArgs {
  const uint8_t* x;
  const uint8_t* x_scale;
  const uint8_t* w;
  const uint8_t* w_scale;
  const float* bias;
  void* y;
  int64_t ldw, block_tiles;
  int N;
  int blocks;  // of 32 columns
  int bytes;   // of a row's codes
  int act, y_bf16;
};

// Eight codes as twice their values.
__device__ __forceinline__ void doubled(uint32_t codes, uint32_t (&v)[2]) {
  const uint32_t at = codes & 0x77777777u, sign = 0x32103210u | (codes >> 1 & 0x44444444u);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t pos = __byte_perm(0x03020100u, 0x0c080604u, at >> (16 * h));
    const uint32_t neg = __byte_perm(0xfdfeff00u, 0xf4f8fafcu, at >> (16 * h));
    v[h] = __byte_perm(pos, neg, sign >> (16 * h));
  }
}

// Four codes' doubled magnitudes; zero where a code's sign bit is set (the permutation then
// gives the sign of the byte).
__device__ __forceinline__ uint32_t looked_up(uint32_t codes) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(0x03020100u), "r"(0x0c080604u), "r"(codes));
  return r;
}

// sum and less grow by the positive and the negative ones of eight codes times x.
__device__ __forceinline__ int dot8(uint32_t codes, const uint32_t (&x)[2], int sum, int& less) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = codes >> (16 * h);
    const uint32_t pos = looked_up(c), neg = looked_up(c ^ 0x8888u);
    sum = __dp4a(static_cast<int>(pos), static_cast<int>(x[h]), sum);
    less = __dp4a(static_cast<int>(neg), static_cast<int>(x[h]), less);
  }
  return sum;
}

// 16 bytes of a row's codes from byte `at` on; zeros past its end (rows start on 16 bytes and
// their pitch is a multiple of it, but what lies past the codes is not theirs).
__device__ __forceinline__ uint4 load_codes(const uint8_t* row, int at, int bytes) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if (at + 16 <= bytes) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(row + at)
                 : "memory");
  } else if (at < bytes) {
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (at + i < bytes) w[i / 4] |= static_cast<uint32_t>(row[at + i]) << (8 * (i % 4));
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

struct PutOne {
  const OneArgs& a;
  int n;
  float sum;
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    put_at<ACT>(static_cast<Out*>(a.y) + n, sum, a.bias != nullptr ? a.bias[n] : 0.f);
  }
};

template <int U, int R>
__global__ void __launch_bounds__(kOneThreads) linear_one_kernel(const OneArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as in the kernel above
  const int lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * (kOneThreads / 32) + (threadIdx.x >> 5)) * R;
  if (n0 >= a.N) return;
  const uint8_t* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = a.w + min(n0 + r, a.N - 1) * a.ldw;
  // R channels from a multiple of R on are 16 bytes apart in a scale tile, those past N too
  static_assert(32 % R == 0, "R channels lie in one 32-row group");
  const uint8_t* ws = a.w_scale + fp4_scale_at(a.block_tiles, n0, 0);
  float acc[R] = {};
  uint32_t top = 0;  // the largest scale byte: whether one is NaN
  for (int b0 = lane; b0 < a.blocks; b0 += 32 * U) {
    uint4 wv[R][U], xv[U];
    uint32_t we[R][U], xe[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * 32;
      const bool in = u == 0 || b < a.blocks;
      const int64_t tile = static_cast<int64_t>(b >> 2) * kFp4Tile + (b & 3);
      xv[u] = load_codes(a.x, b * 16, a.bytes);
      xe[u] = in ? a.x_scale[tile] : 0u;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        wv[r][u] = load_codes(w[r], b * 16, a.bytes);
        we[r][u] = in ? ws[tile + 16 * r] : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t xc[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
      uint32_t x[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) doubled(xc[i], x[i]);
      top = max(top, xe[u]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t wc[4] = {wv[r][u].x, wv[r][u].y, wv[r][u].z, wv[r][u].w};
        int sum = 0, less = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = dot8(wc[i], x[i], sum, less);
        // The sum is four times that of the values. The scales' product in two halves, so
        // that none on the way leaves f32 where the last does not (a half of 2^-127 is
        // taken as zero: the product of both vanishes in f32).
        const uint32_t e = we[r][u] + xe[u], e1 = e >> 1;
        top = max(top, we[r][u]);
        acc[r] += static_cast<float>(sum - less) * 0.25f * __uint_as_float(e1 << 23) *
                  __uint_as_float((e - e1) << 23);
      }
    }
  }
  top = __reduce_max_sync(kFull, top);
  if (top == 255u) {
    // a NaN among the scales (255 + 253 is as well that of two numbers): which of the
    // channels have one
#pragma unroll
    for (int r = 0; r < R; ++r)
      for (int b = lane; b < a.blocks; b += 32)
        if (a.x_scale[fp4_scale_at(a.block_tiles, 0, b)] == 255u ||
            a.w_scale[fp4_scale_at(a.block_tiles, min(n0 + r, a.N - 1), b)] == 255u)
          acc[r] = __uint_as_float(0x7fc00000u);
  }
  float mine = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(kFull, acc[r], o);
    if (lane == r) mine = acc[r];
  }
  if (lane < R && n0 + lane < a.N) by_kind(a, PutOne{a, n0 + lane, mine});
}

constexpr int64_t kMostPitch = int64_t{1} << 40;  // in bytes: tensor maps take less

struct Operands {
  const uint8_t* x;
  const uint8_t* x_scale;
  const uint8_t* w;
  const uint8_t* w_scale;
  int64_t ldx, ldw, M, N, K;
};

// 2-D map of codes {bytes, rows} with the given pitch, box {128, box_rows}, 128-byte
// swizzle; bytes past the matrix read as zero.
cudaError_t encode_codes(CUtensorMap* map, const uint8_t* base, int64_t K, int64_t rows,
                         int64_t ld, int box_rows) {
  const EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>((K + 1) / 2), static_cast<cuuint64_t>(rows)};
  // a single row's pitch leads nowhere, and may be more than a map takes
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? ld : (K + 31) / 32 * 16)};
  const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 3-D map of scale tiles {128 words, tiles along K, row tiles}, box {128, kStageTiles,
// row_tiles}; tiles past the matrix read as zero.
cudaError_t encode_scales(CUtensorMap* map, const uint8_t* base, int64_t K, int64_t rows,
                          int row_tiles) {
  const EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint64_t kt = static_cast<cuuint64_t>(fp4_block_tiles(K));
  const cuuint64_t dims[3] = {kFp4Tile / 4, kt, static_cast<cuuint64_t>((rows + 127) / 128)};
  const cuuint64_t strides[2] = {kFp4Tile, kt * kFp4Tile};
  const cuuint32_t box[3] = {kFp4Tile / 4, kStageTiles, static_cast<cuuint32_t>(row_tiles)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 2-D map of y {N, M}, box {128 bytes, 32 rows}, 128-byte swizzle: a warp's part of it.
cudaError_t encode_out(CUtensorMap* map, const LinArgs& a, int64_t M, int64_t N) {
  const EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint32_t size = a.y_bf16 ? 2 : 4;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldy) * size};
  const cuuint32_t box[2] = {128 / size, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, a.y_bf16 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32,
                         2, a.y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, bool PAIR, int S, bool TOKENS_M>
cudaError_t run_linear(const Operands& op, LinArgs args, int sms, cudaStream_t stream) {
  constexpr bool SPLIT = S > 1;
  using R = Ring<BN, PAIR, TOKENS_M>;
  auto* fn = &linear_fp4_kernel<BN, PAIR, S, TOKENS_M>;
  constexpr int smem = R::kTotal;
  constexpr int kUnitA = (PAIR ? 2 : 1) * kBM;
  // args come with the weights as a
  if (TOKENS_M) std::swap(args.na, args.nb);
  LinMaps maps;
  cudaError_t e = encode_codes(TOKENS_M ? &maps.b : &maps.a, op.w, op.K, op.N, op.ldw,
                               TOKENS_M ? (PAIR ? BN / 2 : BN) : kBM);
  if (e == cudaSuccess)
    e = encode_codes(TOKENS_M ? &maps.a : &maps.b, op.x, op.K, op.M, op.ldx,
                     TOKENS_M ? kBM : (PAIR ? BN / 2 : BN));
  if (e == cudaSuccess)
    e = encode_scales(TOKENS_M ? &maps.sb : &maps.sa, op.w_scale, op.K, op.N,
                      TOKENS_M ? R::kBTiles : 1);
  if (e == cudaSuccess)
    e = encode_scales(TOKENS_M ? &maps.sa : &maps.sb, op.x_scale, op.K, op.M,
                      TOKENS_M ? 1 : R::kBTiles);
  if (TOKENS_M && e == cudaSuccess) e = encode_out(&maps.y, args, op.M, op.N);
  if (e != cudaSuccess) return e;
  // Per device, the instance's shared-memory size is set and (pairs) the
  // resident cluster count asked for once: 0 = not yet, else that count + 1.
  static std::atomic<int> prepared[kMaxDevices];
  int dev = -1;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  const bool cacheable = dev >= 0 && dev < kMaxDevices;
  const int cached = cacheable ? prepared[dev].load(std::memory_order_acquire) : 0;
  if (cached == 0) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  args.tiles_b = (args.nb + BN - 1) / BN;
  args.tiles_a = (args.na + kUnitA - 1) / kUnitA;
  const int64_t tiles = static_cast<int64_t>(args.tiles_a) * args.tiles_b;
  args.tiles = static_cast<int>(tiles);  // no more than of the smallest tiles, which are counted below
  args.by_band = Divisor(static_cast<uint32_t>(args.tiles_a) * kBand);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int64_t grid = std::min<int64_t>(tiles, sms);
  int fit = cached > 0 ? cached - 1 : 0;
  if constexpr (PAIR || SPLIT) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = PAIR ? 2 : S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  if constexpr (PAIR) {
    int pairs = sms / 2;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    if (cached == 0 && cudaOccupancyMaxActiveClusters(&fit, fn, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      fit = 0;
    }
    if (fit > 0) pairs = std::min(pairs, fit);
    grid = 2 * std::min<int64_t>(tiles, pairs);
  }
  if constexpr (SPLIT) grid = tiles * S;
  if (cacheable && cached == 0) prepared[dev].store(fit + 1, std::memory_order_release);
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  return cudaLaunchKernelEx(&cfg, fn, maps, args);
}

template <int U, int R>
cudaError_t run_one(const OneArgs& a, cudaStream_t stream) {
  constexpr int kChannels = kOneThreads / 32 * R;
  return launch(&linear_one_kernel<U, R>, dim3(static_cast<unsigned>((a.N + kChannels - 1) / kChannels)),
                kOneThreads, 0, true, stream, a);
}

// The kernels of the forms and variants in fp4_forms.h, in their order.
template <int I>
cudaError_t run_form(const Operands& op, const LinArgs& a, int sms, cudaStream_t s) {
  constexpr Fp4Form f = kFp4FormOf[I];
  static_assert(f.rows_m == f.units * kBM, "a CTA's channels, or a pair's");
  return run_linear<f.rows_n, f.units == 2, f.split, f.lines>(op, a, sms, s);
}
template <int I>
cudaError_t run_variant(const OneArgs& a, cudaStream_t s) {
  return run_one<kFp4OneOf[I].blocks, kFp4OneOf[I].channels>(a, s);
}
constexpr decltype(&run_form<0>) kRunForm[] = {run_form<0>, run_form<1>, run_form<2>, run_form<3>,
                                               run_form<4>, run_form<5>, run_form<6>, run_form<7>};
constexpr decltype(&run_variant<0>) kRunVariant[] = {run_variant<0>, run_variant<1>, run_variant<2>,
                                                     run_variant<3>, run_variant<4>};
static_assert(sizeof(kRunForm) / sizeof(kRunForm[0]) == kFp4Forms &&
                  sizeof(kRunVariant) / sizeof(kRunVariant[0]) == kFp4Ones,
              "one for each");

cudaError_t launch_linear(const Operands& op, const LinArgs& args, int sms, cudaStream_t s) {
  if (fp4_one_token(op.M, op.N, op.K)) {
    const OneArgs a = {op.x, op.x_scale, op.w, op.w_scale, args.bias, args.y, op.ldw,
                       fp4_block_tiles(op.K), static_cast<int>(op.N),
                       static_cast<int>((op.K + 31) / 32), static_cast<int>((op.K + 1) / 2),
                       args.act, args.y_bf16};
    return kRunVariant[fp4_one(op.N, a.blocks, sms)](a, s);
  }
  const int size = args.y_bf16 ? 2 : 4;
  // whole 16 bytes of a row: the copy engine's stores were seen to end on those, not on elements
  const bool lines = is_aligned(args.y, 16) && args.ldy < kMostPitch / size &&
                     args.ldy * size % 16 == 0 && op.N * size % 16 == 0;
  return kRunForm[fp4_form(op.M, op.N, args.nkb, lines, sms)](op, args, sms, s);
}

}  // namespace
}  // namespace dlrm

extern "C" {

int dlrm_linear_fp4(const uint8_t* x, int64_t ldx, const uint8_t* x_scale, const uint8_t* w,
                    int64_t ldw, const uint8_t* w_scale, const float* bias, int64_t M, int64_t N,
                    int64_t K, int act, void* y, int y_dtype, int64_t ldy, int32_t* status_dev,
                    dlrm_stream_t stream) {
  using namespace dlrm;
  if (act < DLRM_ACT_NONE || act > DLRM_ACT_SIGMOID || !known_dtype(y_dtype)) return DLRM_ERR_ARG;
  // room above M, N and K for the last tile's end
  constexpr int64_t kMost = INT_MAX - 1024;
  if (M < 0 || M > kMost || N < 1 || N > kMost || K < 1 || K > kMost) return DLRM_ERR_SHAPE;
  if (ldx < (K + 1) / 2 || ldw < (K + 1) / 2 || ldy < N) return DLRM_ERR_SHAPE;
  if ((M > 1 && ldx >= kMostPitch) || (N > 1 && ldw >= kMostPitch)) return DLRM_ERR_SHAPE;
  // tiles of the smallest kind, 64 x 128
  if ((M + 63) / 64 * ((N + 127) / 128) > INT_MAX) return DLRM_ERR_SHAPE;
  if (w == nullptr || w_scale == nullptr) return DLRM_ERR_NULL;
  if (M > 0 && (x == nullptr || x_scale == nullptr || y == nullptr)) return DLRM_ERR_NULL;
  if (ldx % 16 != 0 || ldw % 16 != 0 || !is_aligned(x, 16) || !is_aligned(w, 16) ||
      !is_aligned(x_scale, 16) || !is_aligned(w_scale, 16) || !is_aligned(bias, 4) ||
      !is_aligned(y, dtype_size(y_dtype)) || !is_aligned(status_dev, 4))
    return DLRM_ERR_ALIGN;
  if (M == 0) return DLRM_OK;
  const int sms = sm_count_current();
  if (sms == 0) return DLRM_ERR_CUDA;
  LinArgs a = {};
  a.bias = bias;
  a.y = y;
  a.ldy = ldy;
  a.na = static_cast<int>(N);
  a.nb = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.nkb = static_cast<int>((K + kCols - 1) / kCols);
  a.act = act;
  a.y_bf16 = y_dtype == DLRM_TABLE_BF16;
  a.status = status_dev;
  const Operands op = {x, x_scale, w, w_scale, ldx, ldw, M, N, K};
  const auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_linear(op, a, sms, s);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

}  // extern "C"
