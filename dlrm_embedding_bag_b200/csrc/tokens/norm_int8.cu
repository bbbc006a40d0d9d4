// Rows rounded to 8-bit integers with one scale each, after a root-mean-square
// norm of x + residual or as they are (declared in dlrm_int8.h).
//
// With t = h * weight, the normed row is y = t * rstd, so its scale is
// s = rstd * A / 127 with A = max|t|, and y / s = t * 127 / A: the integers do
// not depend on rstd. Sum of squares and maximum are therefore taken in one
// pass over the row, and only the scale waits for the norm.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "common.h"
#include "dlrm_int8.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNormThreads = 512;  // of a row that does not fit registers
constexpr uint32_t kInfBits = 0x7f800000u;
// Below this, a largest value of f32 has others of its row that count among the
// subnormals, and 127 over it leaves f32.
constexpr float kTiny = 1e-30f;

struct NormArgs {
  const void* x;
  const void* residual;  // or null
  const float* weight;   // or null
  void* h_out;           // or null
  int8_t* q;
  float* scale;
  int64_t ldx, ldr, ldh, ldq;
  int M, K;
  float eps;
  int norm;  // 0: the rows as they are (rstd = 1)
};

// Sum and largest bit pattern over the THREADS threads of a row: a warp, or the
// whole block. Every thread gets both.
template <int THREADS>
__device__ __forceinline__ void row_sum_max(float& sum, uint32_t& top) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  top = __reduce_max_sync(kFull, top);
  if constexpr (THREADS > 32) {
    __shared__ float sums[THREADS / 32];
    __shared__ uint32_t tops[THREADS / 32];
    __syncthreads();  // an earlier call's values have been read
    if ((threadIdx.x & 31) == 0) {
      sums[threadIdx.x >> 5] = sum;
      tops[threadIdx.x >> 5] = top;
    }
    __syncthreads();
    // every warp adds the warps' sums, in the same order
    const int w = threadIdx.x & (THREADS / 32 - 1);
    sum = sums[w];
    top = __reduce_max_sync(kFull, tops[w]);
#pragma unroll
    for (int o = THREADS / 64; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
}

// Whether any of the row's threads says so.
template <int THREADS>
__device__ __forceinline__ bool row_any(bool mine) {
  if constexpr (THREADS > 32)
    return __syncthreads_or(mine);
  else
    return __any_sync(kFull, mine);
}

// max(|t|, top), NaN if either is.
__device__ __forceinline__ float max_abs(float top, float t) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(t)));
  return r;
}

// A row's factors: its levels are t * pre * inv, rounded.
struct Levels {
  float pre, inv;
};

// top: bits of max|t|. A row whose maximum is tiny is lifted by a power of two
// first (exact), so that 127 / A stays finite.
__device__ __forceinline__ Levels levels_of(uint32_t top) {
  const float A = __uint_as_float(top);
  Levels f;
  f.pre = A < kTiny ? 0x1p100f : 1.f;
  f.inv = (top == 0 || top >= kInfBits) ? 0.f : __fdiv_rn(127.f, A * f.pre);
  return f;
}

// t * inv rounded to the nearest whole number, ties to even, in the low byte:
// added to 1.5 * 2^23, where a step of f32 is 1, in one fused rounding. (The
// conversion instruction runs at an eighth of this rate.)
__device__ __forceinline__ uint32_t level_bits(float t, float inv) {
  return __float_as_uint(__fmaf_rn(t, inv, 12582912.f));
}

// Chunk of VEC elements of a row at column c: h = x + residual.
template <class T, int VEC>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t m, int c, float (&h)[VEC]) {
  load_f32<T, VEC>(static_cast<const T*>(a.x) + m * a.ldx + c, h);
  if (a.residual != nullptr) {
    float r[VEC];
    load_f32<T, VEC>(static_cast<const T*>(a.residual) + m * a.ldr + c, r);
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] += r[e];
  }
}

template <int VEC>
__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[VEC]) {
  if (a.weight == nullptr) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = 1.f;
  } else if constexpr (VEC == 1) {
    w[0] = __ldg(a.weight + c);
  } else if constexpr (VEC == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2*>(a.weight + c));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.weight + c + e));
      w[e] = v.x, w[e + 1] = v.y, w[e + 2] = v.z, w[e + 3] = v.w;
    }
  }
}

template <int VEC>
__device__ __forceinline__ void store_levels(int8_t* p, float (&t)[VEC], Levels f) {
  if (f.pre != 1.f) {  // the same for the whole row
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] *= f.pre;
  }
  // inv is 0 for a row of zeros, and for one with a NaN or an infinity
  const bool none = f.inv == 0.f;
  if constexpr (VEC == 1) {
    *p = none ? 0 : static_cast<int8_t>(level_bits(t[0], f.inv) & 0xff);
  } else if constexpr (VEC == 2) {
    const uint32_t both =
        __byte_perm(level_bits(t[0], f.inv), level_bits(t[1], f.inv), 0x0040);
    *reinterpret_cast<uint16_t*>(p) = none ? 0 : static_cast<uint16_t>(both);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint32_t lo = __byte_perm(level_bits(t[4 * i], f.inv), level_bits(t[4 * i + 1], f.inv), 0x0040);
      const uint32_t hi = __byte_perm(level_bits(t[4 * i + 2], f.inv), level_bits(t[4 * i + 3], f.inv), 0x0040);
      w[i] = none ? 0u : __byte_perm(lo, hi, 0x5410);
    }
    if constexpr (VEC == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// Sum, maximum and whether any is set, over the THREADS threads of a row, which all get them.
template <int THREADS>
__device__ __forceinline__ void row_join_f64(double& sum, double& top, bool& any) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, o);
    top = fmax(top, __shfl_xor_sync(kFull, top, o));
  }
  any = __any_sync(kFull, any);
  if constexpr (THREADS > 32) {
    __shared__ double sums[THREADS / 32], tops[THREADS / 32];
    __syncthreads();  // an earlier row's values have been read
    if ((threadIdx.x & 31) == 0) {
      sums[threadIdx.x >> 5] = sum;
      tops[threadIdx.x >> 5] = top;
    }
    any = __syncthreads_or(any);
    sum = top = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) {
      sum += sums[w];
      top = fmax(top, tops[w]);
    }
  }
}

// A row in 64 bits, from memory (nothing of it may have been written before): where
// squares or products with the weight leave the range of f32 or vanish in it although
// the normed row need not. In 64 bits neither does: factors of 2^-149 to 2^128.
template <class T, int THREADS>
__device__ __forceinline__ void row_in_f64(const NormArgs& a, int64_t m) {
  const int q = threadIdx.x % THREADS;
  auto load = [&](int c, double& t) {
    float h[1], w[1];
    load_h<T, 1>(a, m, c, h);
    load_weight<1>(a, c, w);
    t = static_cast<double>(h[0]) * w[0];
    return h[0];
  };
  double sum = 0.0, top = 0.0;
  bool bad = false;  // a NaN or an infinity
  for (int c = q; c < a.K; c += THREADS) {
    double t;
    const double h = load(c, t);
    sum += h * h;
    top = fmax(top, fabs(t));
    bad |= !(fabs(t) <= DBL_MAX);
  }
  row_join_f64<THREADS>(sum, top, bad);
  const bool none = bad || top == 0.0;
  if (q == 0)
    a.scale[m] = bad     ? __uint_as_float(0x7fc00000u)
                 : none  ? 0.f
                         : static_cast<float>(top / sqrt(sum / a.K + a.eps) / 127.0);
  const double inv = none ? 0.0 : 127.0 / top;
  for (int c = q; c < a.K; c += THREADS) {
    double t;
    const float h[1] = {load(c, t)};
    if (a.h_out != nullptr) store_f32<T, 1>(static_cast<T*>(a.h_out) + m * a.ldh + c, h);
    a.q[m * a.ldq + c] = none ? 0 : static_cast<int8_t>(__double2int_rn(t * inv));
  }
}

// ... where a block has the row: as a call, with the arguments by value, since its code
// inside a kernel costs the kernel's other rows their registers (6000 rows of 6001 with
// a residual: 106 us so, 162 inside, 170 with the arguments by reference; rows of a
// warp lose nothing by it inside, and 45 against 37 us by a call, 60000 of 250 bf16).
template <class T, int THREADS>
__device__ __noinline__ void block_row_in_f64(const NormArgs a, int64_t m) {
  row_in_f64<T, THREADS>(a, m);
}

// Whether a row is row_in_f64's: the mean of its squares, which are finite numbers or
// more, is above f32 or so small that squares have vanished; or its products with the
// weight have left f32, or are so small that some may have vanished. A row of zeros is
// not: `zeros` tells, asked only where squares and products are all zero.
template <class Zeros>
__device__ __forceinline__ bool is_far(const NormArgs& a, float sum, uint32_t top, Zeros zeros) {
  if (!a.norm) return false;
  if (top >= kInfBits) return a.weight != nullptr;
  if (top == 0 && sum == 0.f) return a.weight != nullptr && !zeros();
  if (a.weight != nullptr && __uint_as_float(top) < kTiny) return true;
  if (top == 0) return false;
  return !(sum + a.eps <= FLT_MAX) || __fmaf_rn(a.eps, static_cast<float>(a.K), sum) < 1e-30f * a.K;
}

// The scale of any other row, from its sum of squares and the bits of max|t|. Two
// divisions and a root: one thread's work, since the levels do not need it.
__device__ __forceinline__ float scale_of(const NormArgs& a, float sum, uint32_t top) {
  if (top >= kInfBits) return __uint_as_float(0x7fc00000u);
  const float A = __uint_as_float(top);
  if (!a.norm || top == 0) return __fdiv_rn(A, 127.f);
  const float mean = __fadd_rn(__fdiv_rn(sum, static_cast<float>(a.K)), a.eps);
  return __fdiv_rn(__fmul_rn(A, __frsqrt_rn(mean)), 127.f);
}

// Blocks of an SM that the compiler leaves registers for, where it would take some
// more: the work around a row's barriers is what its time goes into, and other rows
// cover it. 16 elements a thread: 1280 threads an SM, or 1536 of rows that take 512
// (8665 rows of 6924 f32: 86 us with 1024, 70 so). 32 elements: 1024 threads (8000
// rows of 8192 bf16 with their values written out: 103 us as the compiler chooses, 96
// so), but with a residual the loads that all the registers keep in flight are worth
// more (16384 rows of 4096: 116 us, and 123).
template <int VEC, int TPR, int CH, bool RES>
constexpr int kBlocksAnSM = CH == 1 || TPR > 512 ? 1
                            : VEC * CH > 16      ? (RES ? 1 : 1024 / (TPR < 128 ? 128 : TPR))
                            : TPR == 512         ? (RES ? 2 : 3)
                                                 : 1280 / (TPR < 128 ? 128 : TPR);

// Rows that fit the registers of TPR threads (a warp, or a block), CH chunks of VEC
// elements each: read once, 128 bits a load where rows allow that. Bound by the
// memory: 16384 rows of 4096 bf16 with a residual move 470 MB in 73 us.
template <class T, int VEC, int TPR, int CH, bool RES>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, kBlocksAnSM<VEC, TPR, CH, RES>)
    norm_row_kernel(const NormArgs a) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;  // rows of a block
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (m >= a.M) return;  // whole warps, and only where a row is a warp's
  const int q = threadIdx.x % TPR;
  // all of the row's loads first
  Raw<T, VEC> xs[CH], rs[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * TPR + q) * VEC;
    xs[i] = rs[i] = Raw<T, VEC>();
    if (c < a.K) {
      xs[i] = *reinterpret_cast<const Raw<T, VEC>*>(static_cast<const T*>(a.x) + m * a.ldx + c);
      if constexpr (RES)
        rs[i] = *reinterpret_cast<const Raw<T, VEC>*>(static_cast<const T*>(a.residual) + m * a.ldr + c);
    }
  }
  float h[CH][VEC];
  float sum = 0.f, most = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * TPR + q) * VEC;
    widen<T, VEC>(xs[i], h[i]);
    if constexpr (RES) {
      float r[VEC];
      widen<T, VEC>(rs[i], r);
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[i][e] += r[e];
    }
    if (c < a.K) {
      float w[VEC];
      load_weight<VEC>(a, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum += h[i][e] * h[i][e];
        most = max_abs(most, h[i][e] * w[e]);
      }
    }
  }
  uint32_t top = __float_as_uint(most);
  row_sum_max<TPR>(sum, top);
  const bool far = is_far(a, sum, top, [&] {
    bool any = false;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) any |= h[i][e] != 0.f;  // past the row: 0
    return !row_any<TPR>(any);
  });
  if (far) {  // the same for the whole row
    if constexpr (TPR > 32)
      block_row_in_f64<T, TPR>(a, m);
    else
      row_in_f64<T, TPR>(a, m);
    return;
  }
  if (q == 0) a.scale[m] = scale_of(a, sum, top);
  const Levels f = levels_of(top);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * TPR + q) * VEC;
    if (c < a.K) {
      if (a.h_out != nullptr) store_f32<T, VEC>(static_cast<T*>(a.h_out) + m * a.ldh + c, h[i]);
      float w[VEC];
      load_weight<VEC>(a, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] *= h[i][e];
      store_levels<VEC>(a.q + m * a.ldq + c, w, f);
    }
  }
}

// Longer rows: a block for each row, which it reads twice (the second time from L2).
template <class T, int VEC>
__global__ void __launch_bounds__(kNormThreads)
    norm_loop_kernel(const NormArgs a) {
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    float sum = 0.f, most = 0.f;
    for (int c = threadIdx.x * VEC; c < a.K; c += kNormThreads * VEC) {
      float h[VEC], w[VEC];
      load_h<T, VEC>(a, m, c, h);
      load_weight<VEC>(a, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum += h[e] * h[e];
        most = max_abs(most, h[e] * w[e]);
      }
    }
    uint32_t top = __float_as_uint(most);
    row_sum_max<kNormThreads>(sum, top);
    const bool far = is_far(a, sum, top, [&] {
      bool any = false;
      for (int c = threadIdx.x * VEC; c < a.K; c += kNormThreads * VEC) {
        float h[VEC];
        load_h<T, VEC>(a, m, c, h);
#pragma unroll
        for (int e = 0; e < VEC; ++e) any |= h[e] != 0.f;
      }
      return !row_any<kNormThreads>(any);
    });
    if (far) {
      block_row_in_f64<T, kNormThreads>(a, m);
      continue;
    }
    if (threadIdx.x == 0) a.scale[m] = scale_of(a, sum, top);
    const Levels f = levels_of(top);
    for (int c = threadIdx.x * VEC; c < a.K; c += kNormThreads * VEC) {
      float h[VEC], w[VEC];
      load_h<T, VEC>(a, m, c, h);
      load_weight<VEC>(a, c, w);
      if (a.h_out != nullptr) store_f32<T, VEC>(static_cast<T*>(a.h_out) + m * a.ldh + c, h);
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] *= w[e];
      store_levels<VEC>(a.q + m * a.ldq + c, h, f);
    }
  }
}

template <class T, int VEC>
cudaError_t run_loop(const NormArgs& a, cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>(a.M, kSms * 64);
  return launch(&norm_loop_kernel<T, VEC>, dim3(static_cast<unsigned>(blocks)), kNormThreads, 0,
                false, stream, a);
}

template <class T, int VEC, int TPR, int CH>
cudaError_t run_row(const NormArgs& a, cudaStream_t stream) {
  constexpr int kThreads = TPR < 128 ? 128 : TPR, kRows = kThreads / TPR;
  const int64_t blocks = (static_cast<int64_t>(a.M) + kRows - 1) / kRows;
  auto* fn = a.residual != nullptr ? &norm_row_kernel<T, VEC, TPR, CH, true>
                                   : &norm_row_kernel<T, VEC, TPR, CH, false>;
  return launch(fn, dim3(static_cast<unsigned>(blocks)), kThreads, 0, false, stream, a);
}

// Rows that 128-bit accesses cannot walk: pairs or single elements, eight a thread.
// (30000 rows with a residual and their values written out, f32: 260 us in the
// loop below, here 101 at 1002 columns and 113 at 1001; bf16 253, 94 and 107. The norm
// alone: 75 and 80 us f32, 66 and 76 bf16.)
template <class T, int VEC>
cudaError_t run_narrow(const NormArgs& a, cudaStream_t stream) {
  const int chunks = a.K / VEC;
  if (chunks <= 128) return run_row<T, VEC, 32, 4>(a, stream);
  if (chunks <= 256) return run_row<T, VEC, 32, 8>(a, stream);
  if (chunks <= 1024) return run_row<T, VEC, 128, 8>(a, stream);
  if (chunks <= 2048) return run_row<T, VEC, 256, 8>(a, stream);
  if (chunks <= 4096) return run_row<T, VEC, 512, 8>(a, stream);
  // 1024 threads leave an SM one block, whose barriers nothing covers: 6000 rows of
  // 6001 took 173 to 192 us with eight elements a thread, 123 to 153 with 512 and 16.
  if constexpr (VEC == 1) {
    if (chunks <= 8192) return run_row<T, VEC, 512, 16>(a, stream);
  } else {
    if (chunks <= 8192) return run_row<T, VEC, 1024, 8>(a, stream);
  }
  return run_loop<T, VEC>(a, stream);
}

// Four chunks a thread where rows are many (a row's loads all in flight, many
// rows an SM); one where they are few and a row's latency is what counts.
template <class T>
cudaError_t run_norm(const NormArgs& a, int vec, cudaStream_t stream) {
  constexpr int V = kVecOf<T>;
  if (vec == 1) return run_narrow<T, 1>(a, stream);
  if (vec == 2) return run_narrow<T, 2>(a, stream);
  const int chunks = a.K / V;
  const bool few = a.M <= kSms * 4;
  if (chunks <= 32) return run_row<T, V, 32, 1>(a, stream);
  if (chunks <= 128) return few ? run_row<T, V, 128, 1>(a, stream) : run_row<T, V, 32, 4>(a, stream);
  if (chunks <= 512)
    return few ? run_row<T, V, 512, 1>(a, stream) : run_row<T, V, 128, 4>(a, stream);
  if (chunks <= 1024)
    return few ? run_row<T, V, 1024, 1>(a, stream) : run_row<T, V, 256, 4>(a, stream);
  if (chunks <= 2048) return run_row<T, V, 512, 4>(a, stream);
  if (chunks <= 4096) return run_row<T, V, 1024, 4>(a, stream);
  return run_loop<T, V>(a, stream);
}

int norm_rows(const NormArgs& a, int dtype, cudaStream_t stream) {
  const int es = dtype_size(dtype);
  // elements of an access that every row allows
  int vec = 1;
  for (int v : {2, 16 / es})
    if (a.K % v == 0 && rows_by(a.x, a.ldx, es, v) &&
        (a.residual == nullptr || rows_by(a.residual, a.ldr, es, v)) &&
        (a.h_out == nullptr || rows_by(a.h_out, a.ldh, es, v)) &&
        is_aligned(a.weight, v == 2 ? 8 : 16) && rows_by(a.q, a.ldq, 1, v))
      vec = v;
  using B = __nv_bfloat16;
  cudaError_t e;
  if (dtype == DLRM_TABLE_F32)
    e = run_norm<float>(a, vec, stream);
  else
    e = run_norm<B>(a, vec, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

int check_rows(const void* x, int64_t ldx, int dtype, int64_t M, int64_t K, const int8_t* q,
               int64_t ldq, const float* scale) {
  if (!known_dtype(dtype)) return DLRM_ERR_ARG;
  if (M < 0 || M > INT_MAX || K < 1 || K > INT_MAX - 65536 || ldx < K || ldq < K)
    return DLRM_ERR_SHAPE;
  if (M > 0 && (x == nullptr || q == nullptr || scale == nullptr)) return DLRM_ERR_NULL;
  if (!is_aligned(x, dtype_size(dtype)) || !is_aligned(scale, 4)) return DLRM_ERR_ALIGN;
  return DLRM_OK;
}

// y = q * scale: a block walks rows. VEC 16: one 128-bit load a thread; else four
// accesses of VEC columns a thread, a block's width apart.
template <class T, int VEC>
__global__ void __launch_bounds__(256)
    dequant_kernel(const int8_t* q, int64_t ldq, const float* scale, int M, int K, T* y,
                   int64_t ldy) {
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const float s = __ldg(scale + m);
    const int8_t* from = q + m * ldq;
    T* to = y + m * ldy;
    if constexpr (VEC == 16) {
      for (int c = threadIdx.x * 16; c < K; c += blockDim.x * 16) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(from + c));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = static_cast<float>(static_cast<int8_t>(w[2 * i + e / 4] >> (8 * (e % 4)))) * s;
          store_f32<T, 8>(to + c + 8 * i, v);
        }
      }
    } else {
      const int step = blockDim.x * VEC;
      for (int c0 = threadIdx.x * VEC; c0 < K; c0 += 4 * step) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + i * step;
          r[i] = 0;
          if (c < K) {
            if constexpr (VEC == 4)
              r[i] = __ldg(reinterpret_cast<const uint32_t*>(from + c));
            else if constexpr (VEC == 2)
              r[i] = __ldg(reinterpret_cast<const unsigned short*>(from + c));
            else
              r[i] = static_cast<uint8_t>(__ldg(from + c));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + i * step;
          float v[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            v[e] = static_cast<float>(static_cast<int8_t>(r[i] >> (8 * e))) * s;
          if (c < K) store_f32<T, VEC>(to + c, v);
        }
      }
    }
  }
}

template <class T>
cudaError_t run_dequant(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int64_t K,
                        T* y, int64_t ldy, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(M, kSms * 64));
  int vec = 1;
  for (int v : {2, 4, 16})
    if (K % v == 0 && rows_by(q, ldq, 1, v) && rows_by(y, ldy, sizeof(T), v)) vec = v;
  const int64_t per_row = vec == 16 ? K / 16 : (K / vec + 3) / 4;
  const int threads = static_cast<int>(std::min<int64_t>(256, (per_row + 31) / 32 * 32));
  auto* fn = vec == 16  ? &dequant_kernel<T, 16>
             : vec == 4 ? &dequant_kernel<T, 4>
             : vec == 2 ? &dequant_kernel<T, 2>
                        : &dequant_kernel<T, 1>;
  return launch(fn, dim3(blocks), threads, 0, false, stream, q, ldq, scale, static_cast<int>(M),
                static_cast<int>(K), y, ldy);
}

}  // namespace
}  // namespace dlrm

extern "C" {

int dlrm_rms_norm_int8(const void* x, int64_t ldx, const void* residual, int64_t ldr, int dtype,
                       const float* weight, int64_t M, int64_t K, float eps, void* h_out,
                       int64_t ldh, int8_t* q, int64_t ldq, float* scale, dlrm_stream_t stream) {
  using namespace dlrm;
  int rc = check_rows(x, ldx, dtype, M, K, q, ldq, scale);
  if (rc != DLRM_OK) return rc;
  if ((residual != nullptr && ldr < K) || (h_out != nullptr && ldh < K)) return DLRM_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > FLT_MAX) return DLRM_ERR_ARG;
  const int es = dtype_size(dtype);
  if (!is_aligned(residual, es) || !is_aligned(h_out, es) || !is_aligned(weight, 4))
    return DLRM_ERR_ALIGN;
  if (M == 0) return DLRM_OK;
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h_out = h_out;
  a.q = q;
  a.scale = scale;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.ldq = ldq;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  a.eps = eps;
  a.norm = 1;
  return norm_rows(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int dlrm_quantize_int8(const void* x, int64_t ldx, int dtype, int64_t M, int64_t K, int8_t* q,
                       int64_t ldq, float* scale, dlrm_stream_t stream) {
  using namespace dlrm;
  int rc = check_rows(x, ldx, dtype, M, K, q, ldq, scale);
  if (rc != DLRM_OK || M == 0) return rc;
  NormArgs a = {};
  a.x = x;
  a.q = q;
  a.scale = scale;
  a.ldx = ldx;
  a.ldq = ldq;
  a.M = static_cast<int>(M);
  a.K = static_cast<int>(K);
  return norm_rows(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int dlrm_dequantize_int8(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int64_t K,
                         void* y, int dtype, int64_t ldy, dlrm_stream_t stream) {
  using namespace dlrm;
  int rc = check_rows(y, ldy, dtype, M, K, q, ldq, scale);
  if (rc != DLRM_OK || M == 0) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == DLRM_TABLE_F32
          ? run_dequant(q, ldq, scale, M, K, static_cast<float*>(y), ldy, s)
          : run_dequant(q, ldq, scale, M, K, static_cast<__nv_bfloat16*>(y), ldy, s);
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

}  // extern "C"
