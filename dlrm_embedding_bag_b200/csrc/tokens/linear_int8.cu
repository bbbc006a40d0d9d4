// The layer on 8-bit integers (declared in dlrm_int8.h):
// y[m][n] = act(x_scale[m] * w_scale[n] * sum_k x[m][k] w[n][k] + bias[n]).
//
// The weights take the tensor cores' M side and the tokens their N side, so an
// accumulator lane is an output channel and a column a token: the scale and
// the bias of a channel stay in its lane's registers, the 32 lanes of a warp
// write 32 neighbouring channels of one token without staging (whole sectors where
// base and pitch are multiples of 32 bytes, else one more sector a store, two of them
// in part), and few tokens make a narrow tile instead of a mostly empty one.
//
// Ten warps a CTA, as in the bf16 layer (linear.cu): one thread streams 128-byte
// K blocks of both operands into a shared-memory ring with 2-D TMA loads, one
// issues tcgen05.mma.kind::i8 (K = 32 each, int32 sums in TMEM, two
// accumulators), eight warps drain a finished accumulator while the next tile's
// products fill the other. Three forms:
//   - one CTA walks 128-channel x BN-token tiles;
//   - CTA pairs (cta_group::2) walk 256 x 256 tiles, each CTA loading its 128
//     channels and half of the tokens;
//   - few tiles: a cluster of S CTAs shares one tile, each summing a stretch of
//     K; the int32 parts meet through distributed shared memory (exact, so the
//     split changes no bit).
// Every wait is bounded; one that runs out sets DLRM_FLAG_TIMEOUT in the
// optional status word, and the CTA still lets its loads land, frees its tensor
// memory and exits.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>

#include "common.h"
#include "dlrm_int8.h"
#include "ring_landing.h"
#include "tcgen05_common.cuh"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBM = 128;  // channels of a CTA's tile
constexpr int kBK = 128;  // bytes of K per stage: one 128-byte swizzle row
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr long long kWaitLimit = 200000000LL;  // clock cycles, about 0.1 s
constexpr int kMaxDevices = 64;                // devices whose launch set-up is cached

struct LinArgs {
  const float* x_scale;
  const float* w_scale;
  const float* bias;
  void* y;
  int64_t ldy;
  int M, N;
  int nkb;                       // K blocks
  int tiles_m, tiles_n, tiles;   // token tiles, channel tiles
  int act, y_bf16;
  int32_t* status;
};

struct alignas(64) LinMaps {
  CUtensorMap w, x;
};

template <int BN, bool PAIR>
struct Ring {
  static constexpr int kW = kBM * kBK;
  static constexpr int kX = (PAIR ? BN / 2 : BN) * kBK;
  static constexpr int kStage = kW + kX;
  // as many stages as fit in about 192 KB, at most 8
  static constexpr int kStages = (192 * 1024 / kStage) < 8 ? (192 * 1024 / kStage) : 8;
  static constexpr int kScales = kStages * kStage;  // x_scale of a tile, a slice per warp
  static constexpr int kBars = kScales + kEpiWarps * (BN / 2 < 32 ? 32 : BN / 2) * 4;
  static constexpr int kTotal = kBars + (2 * kStages + 5) * 8 + 8 + 1024;  // + alignment
  static_assert(kTotal <= 227 * 1024, "shared memory of one CTA");
};

// Instruction descriptor of tcgen05.mma.kind::i8 with signed 8-bit A and B, both
// K-major, wrapping int32 sums, dense, shape M x N: D format S32 (bits 4-5 = 2),
// A and B signed (7-9 = 1, 10-12 = 1), N >> 3 (17-22), M >> 4 (24-28).
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T for one K = 32 step of 8-bit integers.
template <int CG>
__device__ __forceinline__ void tc_mma_s8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint4 load_cluster_v4(uint32_t cluster_addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
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

// An output channel's constants and its column of y.
struct Channel {
  float ws, b;
  bool live;
};

// One output from its int32 sum, the same in every form of the layer: two
// roundings, the sum's own and a product's, then one fused with the bias.
template <int ACT, class Out>
__device__ __forceinline__ void put_at(Out* p, const Channel& ch, int sum, float xs) {
  const float v = activate<ACT>(__fmaf_rn(__fmul_rn(static_cast<float>(sum), xs), ch.ws, ch.b));
  if constexpr (sizeof(Out) == 4)
    *p = v;
  else
    *p = __float2bfloat16_rn(v);
}

template <int ACT, class Out>
__device__ __forceinline__ void put(const LinArgs& a, const Channel& ch, int n, int m, int sum,
                                    float xs) {
  put_at<ACT>(static_cast<Out*>(a.y) + static_cast<int64_t>(m) * a.ldy + n, ch, sum, xs);
}

// One warp's share of a finished accumulator: 32 channels (its TMEM lanes),
// tokens m0 + c for the columns c of [c0, c1). The address walks from token to
// token: a 64-bit product for each made it 19 instructions an element.
template <int ACT, class Out>
__device__ __forceinline__ void drain(const LinArgs& a, const Channel& ch, int n, int m0,
                                      const float* xs, uint32_t tmem, int c0, int c1) {
  Out* p = static_cast<Out*>(a.y) + static_cast<int64_t>(m0 + c0) * a.ldy + n;
  for (int c = c0; c < c1 && m0 + c < a.M; c += 32) {
    float v[32];
    tmem_ld_32x32b_x32(tmem + c, v);
    const int left = a.M - (m0 + c);
    const float4* s = reinterpret_cast<const float4*>(xs + (c - c0));
    if (!ch.live) {
      // a channel past N: nothing to write
    } else if (left >= 32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 f = s[i];
        put_at<ACT>(p, ch, __float_as_int(v[4 * i]), f.x);
        p += a.ldy;
        put_at<ACT>(p, ch, __float_as_int(v[4 * i + 1]), f.y);
        p += a.ldy;
        put_at<ACT>(p, ch, __float_as_int(v[4 * i + 2]), f.z);
        p += a.ldy;
        put_at<ACT>(p, ch, __float_as_int(v[4 * i + 3]), f.w);
        p += a.ldy;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i < left) put_at<ACT>(p, ch, __float_as_int(v[i]), xs[c - c0 + i]);
        p += a.ldy;
      }
    }
    __syncwarp();  // the next load takes the whole warp
  }
}

// Calls f with the activation and the output type as types.
template <class F>
__device__ __forceinline__ void by_kind(const LinArgs& a, F f) {
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

struct DrainCall {
  const LinArgs& a;
  const Channel& ch;
  int n, m0;
  const float* xs;
  uint32_t tmem;
  int c0, c1;
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    drain<ACT, Out>(a, ch, n, m0, xs, tmem, c0, c1);
  }
};

// The cluster's parts of a tile, kept as [column][channel] int32 at the start
// of each CTA's ring, summed over its S CTAs for columns [c0, c1): a column's
// 128 channels a warp, four a lane, the loads of eight parts in flight. (One
// 4-byte load after another, an earlier form, took 5 us of a 10 us layer.)
template <int S>
struct JoinCall {
  const LinArgs& a;
  int n0, m0, c0, c1, ew, lane;
  uint32_t smem;
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    constexpr int kCols = 8 / S;  // columns at a time
    const int n = n0 + lane * 4;
    Channel ch[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ch[e] = {0.f, 0.f, n + e < a.N};
      if (ch[e].live) {
        ch[e].ws = a.w_scale[n + e];
        ch[e].b = a.bias != nullptr ? a.bias[n + e] : 0.f;
      }
    }
    for (int cb = c0 + ew * kCols; cb < c1; cb += kEpiWarps * kCols) {
      uint4 v[kCols][S];
      float xs[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const bool live = cb + i < c1 && m0 + cb + i < a.M;
        xs[i] = live ? a.x_scale[m0 + cb + i] : 0.f;
#pragma unroll
        for (int k = 0; k < S; ++k) {
          v[i][k] = make_uint4(0, 0, 0, 0);
          if (live) v[i][k] = load_cluster_v4(map_to_cta(smem + ((cb + i) * kBM + lane * 4) * 4, k));
        }
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        if (cb + i >= c1 || m0 + cb + i >= a.M) break;
        uint4 t = v[i][0];
#pragma unroll
        for (int k = 1; k < S; ++k)
          t.x += v[i][k].x, t.y += v[i][k].y, t.z += v[i][k].z, t.w += v[i][k].w;
        const uint32_t sums[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (ch[e].live)
            put<ACT, Out>(a, ch[e], n + e, m0 + cb + i, static_cast<int>(sums[e]), xs[i]);
      }
    }
  }
};

// Tile t -> (token tile, channel tile): bands of 8 token tiles, so that the CTAs
// at work at one time read few different rows of either operand.
__device__ __forceinline__ void tile_at(const LinArgs& a, int t, int& tm, int& tn) {
  constexpr int kBand = 8;
  const int per_band = kBand * a.tiles_n;
  const int band = t / per_band, in = t % per_band;
  const int height = min(kBand, a.tiles_m - band * kBand);
  tm = band * kBand + in % height;
  tn = in / height;
}

// S > 1: the S CTAs of a cluster share one tile (and there is one tile a cluster).
template <int BN, bool PAIR, int S>
__global__ void __launch_bounds__(kThreads, 1)
    linear_int8_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinArgs args) {
  constexpr bool SPLIT = S > 1;
  static_assert(!(PAIR && SPLIT), "a pair shares a tile's channels, not its K");
  using R = Ring<BN, PAIR>;
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int kUnitN = CG * kBM;                          // channels of a unit's tile
  constexpr uint32_t kCols = 2 * BN < 32 ? 32 : 2 * BN;     // two accumulators
  constexpr int kWarpCols = BN / 2 < 32 ? 32 : BN / 2;      // columns an epilogue warp drains
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + R::kBars);
  uint64_t* empty = full + R::kStages;
  uint64_t* acc_full = empty + R::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(mma_done + 1);
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
    tmem_alloc<CG>(tslot, kCols);
    tmem_relinquish<CG>();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < R::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], CG * kEpiWarps);
    }
    mbar_init(mma_done, 1);
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
  // Everything below may come from the kernel before (the levels, the scales), which
  // may still be at work, so every role waits for its end. The loads behind the wait
  // are ordinary ones: those of the read-only path (__ldg, .nc) may be moved in front
  // of it, and ask that nothing writes the memory while this kernel runs. This grid lets
  // none start before its own end: the bf16 layers read their bias without waiting.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool timed_out = false;

  if (warp == 0) {
    if (lane == 0) {
      int g = 0;
      for (int t = unit0; t < args.tiles && !timed_out; t += unit_step) {
        int tm, tn;
        tile_at(args, t, tm, tn);
        const int n0 = tn * kUnitN + (PAIR ? static_cast<int>(rank) * kBM : 0);
        const int m0 = tm * BN + (PAIR ? static_cast<int>(rank) * (BN / 2) : 0);
        for (int kb = kb_begin; kb < kb_end; ++kb, ++g) {
          const int s = g % R::kStages;
          if (g >= R::kStages &&
              !mbar_wait_bounded(&empty[s], ((g / R::kStages) - 1) & 1, kWaitLimit)) {
            timed_out = true;
            break;
          }
          uint8_t* sw = smem + s * R::kStage;
          uint8_t* sx = sw + R::kW;
          if constexpr (PAIR) {
            // both CTAs' bytes are counted on the issuer's barrier, which only
            // its producer arms
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * R::kStage);
            const uint32_t fb = map_to_cta(smem_u32(&full[s]), 0);
            tma_load_2d_pair(sw, &maps.w, fb, kb * kBK, n0);
            tma_load_2d_pair(sx, &maps.x, fb, kb * kBK, m0);
          } else {
            mbar_arrive_expect_tx(&full[s], R::kStage);
            tma_load_2d(sw, &maps.w, &full[s], kb * kBK, n0);
            tma_load_2d(sx, &maps.x, &full[s], kb * kBK, m0);
          }
        }
      }
      // no load is in flight once this CTA leaves, whoever gave up
      land_loads<R::kStages, PAIR>(
          !PAIR || rank == 0, timed_out, g,
          [&](int s, uint32_t parity) { (void)mbar_wait_bounded(&full[s], parity, kWaitLimit); },
          [&](int s) { mbar_arrive_expect_tx(&full[s], R::kStage); },
          [&](int steps) { tell_steps(other_steps, steps); },
          [&] { return told_steps(other_steps, (R::kStages + 2) * kWaitLimit); });
    }
  } else if (warp == 1) {
    if (lane == 0 && (!PAIR || rank == 0)) {
      constexpr uint32_t idesc = idesc_s8_s32(kUnitN, BN);
      int g = 0, j = 0;
      for (int t = unit0; t < args.tiles && !timed_out; t += unit_step, ++j) {
        const int b = j & 1;
        if (j >= 2 && !mbar_wait_bounded(&acc_empty[b], ((j >> 1) - 1) & 1, kWaitLimit)) {
          timed_out = true;
          break;
        }
        tc_fence_after_sync();
        const uint32_t acc = tmem + static_cast<uint32_t>(b * BN);
        for (int kb = kb_begin; kb < kb_end; ++kb, ++g) {
          const int s = g % R::kStages;
          if (!mbar_wait_bounded(&full[s], (g / R::kStages) & 1, kWaitLimit)) {
            timed_out = true;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sw = smem_u32(smem + s * R::kStage);
          const uint32_t sx = sw + R::kW;
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            tc_mma_s8<CG>(acc, sdesc_k_sw128(sw + k * 32), sdesc_k_sw128(sx + k * 32), idesc,
                          (kb > kb_begin || k > 0) ? 1u : 0u);
          if constexpr (PAIR)
            tc_commit_pair_both(&empty[s]);
          else
            tc_commit<CG>(&empty[s]);
        }
        if constexpr (PAIR)
          tc_commit_pair_both(&acc_full[b]);
        else
          tc_commit<CG>(&acc_full[b]);
      }
      // every MMA has completed before this CTA or its peer can leave
      tc_commit<CG>(mma_done);
      if (!mbar_wait_bounded(mma_done, 0, kWaitLimit)) timed_out = true;
    }
  } else {
    const int ew = warp - 2, quarter = warp & 3;
    const int c_begin = (ew >> 2) * kWarpCols;
    const int c_end = min(BN, c_begin + kWarpCols);
    float* xs = reinterpret_cast<float*>(smem + R::kScales) + ew * kWarpCols;
    int j = 0;
    for (int t = unit0; t < args.tiles; t += unit_step, ++j) {
      const int b = j & 1;
      int tm, tn;
      tile_at(args, t, tm, tn);
      const int m0 = tm * BN;
      const int n = tn * kUnitN + (PAIR ? static_cast<int>(rank) * kBM : 0) + quarter * 32 + lane;
      Channel ch = {0.f, 0.f, n < args.N};
      if constexpr (!SPLIT) {
        if (ch.live) {
          ch.ws = args.w_scale[n];
          ch.b = args.bias != nullptr ? args.bias[n] : 0.f;
        }
        __syncwarp();  // the slice's readers of the tile before are done
        for (int c = c_begin + lane; c < c_end; c += 32)
          xs[c - c_begin] = m0 + c < args.M ? args.x_scale[m0 + c] : 0.f;
        __syncwarp();
      }
      if (!__all_sync(kFull, mbar_wait_bounded(&acc_full[b], (j >> 1) & 1, kWaitLimit))) {
        timed_out = true;
        break;
      }
      tc_fence_after_sync();
      const uint32_t tq =
          tmem + static_cast<uint32_t>(b * BN) + (static_cast<uint32_t>(quarter * 32) << 16);
      if constexpr (SPLIT) {
        // all products are done: the ring is free for this CTA's part
        int* part = reinterpret_cast<int*>(smem);
        for (int c = c_begin; c < c_end; c += 32) {
          float v[32];
          tmem_ld_32x32b_x32(tq + c, v);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            part[(c + i) * kBM + quarter * 32 + lane] = __float_as_int(v[i]);
        }
      } else {
        by_kind(args, DrainCall{args, ch, n, m0, xs, tq, c_begin, c_end});
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_remote(map_to_cta(smem_u32(&acc_empty[b]), 0));
        else
          mbar_arrive(&acc_empty[b]);
      }
    }
  }
  if (timed_out && args.status != nullptr) atomicOr(args.status, DLRM_FLAG_TIMEOUT);
  if constexpr (SPLIT) {
    cluster_sync();  // every CTA's part is in its shared memory
    if (warp >= 2) {
      int tm, tn;
      tile_at(args, unit0, tm, tn);
      const int c0 = BN * static_cast<int>(rank) / S, c1 = BN * static_cast<int>(rank + 1) / S;
      by_kind(args, JoinCall<S>{args, tn * kBM, tm * BN, c0, c1, warp - 2, lane, smem_u32(smem)});
    }
  }
  tc_fence_before_sync();
  if constexpr (PAIR || SPLIT)
    cluster_sync();  // no CTA leaves while another may still use its memory
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc<CG>(tmem, kCols);
}

// Few tokens: a warp for each R output channels, four products an instruction,
// the weights read once with 128-bit loads past L1 (which the tokens' rows,
// read by every warp, keep), eight in flight a lane. Bound by reading the
// weights, with about 2 us for a launch's latencies around it. Measured on B200
// in a graph, 16 MB of weights from HBM, against the cluster form below: one
// token 5.1 (R = 1, K = 4096; 3.3 TB/s) and 7.9 us, two 6.4 and 8.0, four 8.0
// and 8.3, eight 11.1 and 8.9; 8192 channels of K = 2048 with R = 2: one 5.1
// and 7.6, four 5.8 and 8.1. R = 2 is slower at K = 4096 (6.9 us), R = 1 at K =
// 2048 (5.6 us). (As first built, from which the rules come. Scales and bias loaded
// before the sums are joined: one token 5.4 to 5.6, two 6.8, four 7.8, behind a
// flushed L2 of 16 calls in a graph.)
constexpr int kVecThreads = 256;
constexpr int kFewTokens = 4;

struct VecArgs {
  LinArgs lin;
  const int8_t* x;
  const int8_t* w;
  int64_t ldx, ldw;
  int K;
};

__device__ __forceinline__ uint4 load_once(const int8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int s) {
  s = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), s);
  s = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), s);
  s = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), s);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), s);
}

// A lane's output of the R * MT, if it has one.
struct FewOut {
  Channel ch;
  int n, m;
  float xs;
};

template <int MT, int R>
struct PutCall {
  const VecArgs& a;
  const FewOut& out;
  const int (&acc)[R][MT];
  template <int ACT, class Out>
  __device__ __forceinline__ void run() const {
    int sum = 0;
#pragma unroll
    for (int i = 0; i < R * MT; ++i)
      if ((threadIdx.x & 31) == i) sum = acc[i / MT][i % MT];
    if (out.ch.live) put<ACT, Out>(a.lin, out.ch, out.n, out.m, sum, out.xs);
  }
};

template <int MT, int R>
__global__ void __launch_bounds__(kVecThreads) linear_few_kernel(const VecArgs a) {
  static_assert(MT * R <= 32, "a lane for each output");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // as in the kernel above
  const int lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * (kVecThreads / 32) + (threadIdx.x >> 5)) * R;
  if (n0 >= a.lin.N) return;
  const int8_t* w[R];
  const int8_t* x[MT];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = a.w + min(n0 + r, a.lin.N - 1) * a.ldw;
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = a.x + min(m, a.lin.M - 1) * a.ldx;
  int acc[R][MT] = {};
  constexpr int U = 8 / R;  // K steps in flight
  const int whole = a.K / 16 * 16;
  for (int k0 = lane * 16; k0 < whole; k0 += 512 * U) {
    uint4 wv[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        wv[u][r] = make_uint4(0, 0, 0, 0);
        if (k0 + u * 512 < whole) wv[u][r] = load_once(w[r] + k0 + u * 512);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint4 xv[MT];
      const int k = min(k0 + u * 512, whole - 16);  // past the end: against zeros
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[m] = *reinterpret_cast<const uint4*>(x[m] + k);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][m] = dot16(wv[u][r], xv[m], acc[r][m]);
    }
  }
  // the last K % 16 columns, one a lane
  if (whole + lane < a.K) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int v = w[r][whole + lane];
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[r][m] += v * x[m][whole + lane];
    }
  }
  // the lane's scales and bias, on their way while the sums are joined; every lane
  // loads some, without a branch
  const int i = min(lane, R * MT - 1);
  FewOut out = {{0.f, 0.f, lane < R * MT && n0 + i / MT < a.lin.N && i % MT < a.lin.M},
                min(n0 + i / MT, a.lin.N - 1), min(i % MT, a.lin.M - 1), 0.f};
  out.ch.ws = a.lin.w_scale[out.n];
  if (a.lin.bias != nullptr) out.ch.b = a.lin.bias[out.n];
  out.xs = a.lin.x_scale[out.m];
  __syncwarp();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[r][m] = __reduce_add_sync(kFull, acc[r][m]);
  by_kind(a.lin, PutCall<MT, R>{a, out, acc});
}

// 2-D map of an int8 matrix {K, rows} with the given pitch, box {128, box_rows},
// 128-byte swizzle; elements past the matrix read as zero.
cudaError_t encode_int8(CUtensorMap* map, const int8_t* base, int64_t K, int64_t rows, int64_t ld,
                        int box_rows) {
  const EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Operands {
  const int8_t* x;
  const int8_t* w;
  int64_t ldx, ldw, K;
};

template <int BN, bool PAIR, int S>
cudaError_t run_linear(const Operands& op, LinArgs args, int sms, cudaStream_t stream) {
  constexpr bool SPLIT = S > 1;
  auto* fn = &linear_int8_kernel<BN, PAIR, S>;
  constexpr int smem = Ring<BN, PAIR>::kTotal;
  constexpr int kUnitN = (PAIR ? 2 : 1) * kBM;
  LinMaps maps;
  cudaError_t e = encode_int8(&maps.w, op.w, op.K, args.N, op.ldw, kBM);
  if (e == cudaSuccess)
    e = encode_int8(&maps.x, op.x, op.K, args.M, op.ldx, PAIR ? BN / 2 : BN);
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
  args.tiles_m = (args.M + BN - 1) / BN;
  args.tiles_n = (args.N + kUnitN - 1) / kUnitN;
  const int64_t tiles = static_cast<int64_t>(args.tiles_m) * args.tiles_n;
  if (tiles > INT_MAX || static_cast<int64_t>(args.tiles_n) * 8 > INT_MAX)
    return cudaErrorInvalidValue;
  args.tiles = static_cast<int>(tiles);
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

template <int MT, int R>
cudaError_t run_few(const Operands& op, const LinArgs& args, cudaStream_t stream) {
  const VecArgs a = {args, op.x, op.w, op.ldx, op.ldw, static_cast<int>(op.K)};
  constexpr int kChannels = kVecThreads / 32 * R;
  return launch(&linear_few_kernel<MT, R>, dim3((args.N + kChannels - 1) / kChannels), kVecThreads,
                0, true, stream, a);
}

// The forms of the tensor-core kernel, with what they take on a B200 in us: a K
// block of 128 bytes of a tile (`step`; much the same for 20 and for 48 KB, so it is
// neither the loads' bytes nor the products but what a stage costs besides: a wait,
// arming and two loads in one thread, a wait, four products and a commit in another),
// what a tile takes besides (`tile`), the least that a tile takes
// (`least`: its drain), and the joining of a cluster's parts (`join`). Fitted to
// all forms at 27 shapes from 5 x 512 x 512 to 65536 x 512 x 592 in a graph; the
// choice was the fastest form, or within 5 % of it, at 26 of them.
struct Form {
  int bn;
  bool pair;
  int split;
  double step, tile, least, join;
  cudaError_t (*run)(const Operands&, LinArgs, int, cudaStream_t);
};
const Form kForms[] = {
    {32, false, 1, 0.285, 0.5, 0.0, 0.0, run_linear<32, false, 1>},
    {32, false, 2, 0.285, 0.5, 0.0, 1.5, run_linear<32, false, 2>},
    {32, false, 4, 0.285, 0.5, 0.0, 2.2, run_linear<32, false, 4>},
    {64, false, 1, 0.290, 0.7, 0.0, 0.0, run_linear<64, false, 1>},
    {64, false, 2, 0.290, 0.7, 0.0, 1.7, run_linear<64, false, 2>},
    {64, false, 4, 0.290, 0.7, 0.0, 2.4, run_linear<64, false, 4>},
    {128, false, 1, 0.280, 1.2, 2.0, 0.0, run_linear<128, false, 1>},
    {128, false, 2, 0.280, 1.2, 2.0, 2.7, run_linear<128, false, 2>},
    {128, false, 4, 0.280, 1.2, 2.0, 3.0, run_linear<128, false, 4>},
    {256, false, 1, 0.320, 2.3, 3.6, 0.0, run_linear<256, false, 1>},
    {256, true, 1, 0.310, 2.2, 3.7, 0.0, run_linear<256, true, 1>},
};

// Few tokens take the kernel for them; the others the form that takes the least
// time by the figures above.
cudaError_t launch_linear(const Operands& op, const LinArgs& args, int sms, cudaStream_t s) {
  if (args.M <= kFewTokens) {
    const bool two = op.K <= 2048;  // channels a warp
    if (args.M == 1) return two ? run_few<1, 2>(op, args, s) : run_few<1, 1>(op, args, s);
    if (args.M == 2) return two ? run_few<2, 2>(op, args, s) : run_few<2, 1>(op, args, s);
    return two ? run_few<4, 2>(op, args, s) : run_few<4, 1>(op, args, s);
  }
  Form best = {};
  double least = 0;
  for (const Form& f : kForms) {
    const int64_t channels = f.pair ? 2 * kBM : kBM;
    const int64_t tiles = (static_cast<int64_t>(args.M) + f.bn - 1) / f.bn *
                          ((static_cast<int64_t>(args.N) + channels - 1) / channels);
    // a cluster's CTAs run at the same time, and each has two K blocks at least
    if (f.split > 1 && (tiles * f.split > 128 || args.nkb < 2 * f.split)) continue;
    const int64_t units = f.pair ? sms / 2 : sms;
    const int64_t rounds = (tiles + units - 1) / units;
    const double us =
        rounds * std::max(f.least, f.step * args.nkb / f.split + f.tile) + f.join;
    if (best.run == nullptr || us < least) {
      best = f;
      least = us;
    }
  }
  return best.run(op, args, sms, s);
}

}  // namespace
}  // namespace dlrm

extern "C" {

int dlrm_linear_int8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                     int64_t ldw, const float* w_scale, const float* bias, int64_t M, int64_t N,
                     int64_t K, int act, void* y, int y_dtype, int64_t ldy, int32_t* status_dev,
                     dlrm_stream_t stream) {
  using namespace dlrm;
  if (act < DLRM_ACT_NONE || act > DLRM_ACT_SIGMOID || !known_dtype(y_dtype)) return DLRM_ERR_ARG;
  // room above M and N for the last tile's end
  if (M < 0 || M > INT_MAX - 1024 || N < 1 || N > INT_MAX - 1024 || K < 1 ||
      K > DLRM_INT8_MAX_K)
    return DLRM_ERR_SHAPE;
  if (ldx < K || ldw < K || ldy < N) return DLRM_ERR_SHAPE;
  if (w == nullptr || w_scale == nullptr) return DLRM_ERR_NULL;
  if (M > 0 && (x == nullptr || x_scale == nullptr || y == nullptr)) return DLRM_ERR_NULL;
  if (ldx % 16 != 0 || ldw % 16 != 0 || !is_aligned(x, 16) || !is_aligned(w, 16) ||
      !is_aligned(x_scale, 4) || !is_aligned(w_scale, 4) || !is_aligned(bias, 4) ||
      !is_aligned(y, dtype_size(y_dtype)) || !is_aligned(status_dev, 4))
    return DLRM_ERR_ALIGN;
  if (M == 0) return DLRM_OK;
  const int sms = sm_count_current();
  if (sms == 0) return DLRM_ERR_CUDA;
  LinArgs a = {};
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.y = y;
  a.ldy = ldy;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.nkb = static_cast<int>((K + kBK - 1) / kBK);
  a.act = act;
  a.y_bf16 = y_dtype == DLRM_TABLE_BF16;
  a.status = status_dev;
  const Operands op = {x, w, ldx, ldw, K};
  const cudaError_t e = launch_linear(op, a, sms, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

}  // extern "C"
