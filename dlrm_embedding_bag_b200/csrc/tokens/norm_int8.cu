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
constexpr int kNormThreads = 256;
constexpr uint32_t kInfBits = 0x7f800000u;

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

// Sum and largest bit pattern over the block; every thread gets both.
template <int THREADS>
__device__ __forceinline__ void block_sum_max(float& sum, uint32_t& top) {
  __shared__ float sums[THREADS / 32];
  __shared__ uint32_t tops[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  top = __reduce_max_sync(kFull, top);
  if constexpr (THREADS > 32) {
    __syncthreads();  // an earlier call's values have been read
    if ((threadIdx.x & 31) == 0) {
      sums[threadIdx.x >> 5] = sum;
      tops[threadIdx.x >> 5] = top;
    }
    __syncthreads();
    sum = 0.f;
    top = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      sum += sums[w];
      top = max(top, tops[w]);
    }
  }
}

// |t|'s bits: as unsigned numbers they order like |t|, infinities and NaNs last.
__device__ __forceinline__ uint32_t abs_bits(float t) { return __float_as_uint(t) & 0x7fffffffu; }

// A row's factors: q = rint(t * pre * inv).
struct Levels {
  float pre, inv;
};

// top: bits of max|t|. A row whose maximum is tiny is lifted by a power of two
// first (exact), so that 127 / A stays finite.
__device__ __forceinline__ Levels levels_of(uint32_t top) {
  const float A = __uint_as_float(top);
  Levels f;
  f.pre = A < 1e-30f ? 0x1p100f : 1.f;
  f.inv = (top == 0 || top >= kInfBits) ? 0.f : __fdiv_rn(127.f, A * f.pre);
  return f;
}

__device__ __forceinline__ int8_t level(float t, Levels f) {
  // f.inv is 0 for a row of zeros and for one with a NaN or an infinity: 0
  return f.inv == 0.f ? 0 : static_cast<int8_t>(__float2int_rn(t * f.pre * f.inv));
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
  } else {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.weight + c + e));
      w[e] = v.x, w[e + 1] = v.y, w[e + 2] = v.z, w[e + 3] = v.w;
    }
  }
}

template <int VEC>
__device__ __forceinline__ void store_levels(int8_t* p, const float (&t)[VEC], Levels f) {
  if constexpr (VEC == 1) {
    *p = level(t[0], f);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      w[i] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(level(t[4 * i + e], f))) << (8 * e);
    }
    if constexpr (VEC == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// The squares of a row left the range of f32 (or vanished in it) although the
// row itself did not: its scale from squares of h / max|h|. Reads the row
// again, before anything of it is written.
template <class T, int VEC, int THREADS>
__device__ float far_scale(const NormArgs& a, int64_t m, uint32_t top) {
  float none = 0.f, sum = 0.f;
  uint32_t hbits = 0;
  for (int c = threadIdx.x * VEC; c < a.K; c += THREADS * VEC) {
    float h[VEC];
    load_h<T, VEC>(a, m, c, h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) hbits = max(hbits, abs_bits(h[e]));
  }
  block_sum_max<THREADS>(none, hbits);
  const float big = __uint_as_float(hbits);
  for (int c = threadIdx.x * VEC; c < a.K; c += THREADS * VEC) {
    float h[VEC];
    load_h<T, VEC>(a, m, c, h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float s = __fdiv_rn(h[e], big);
      sum += s * s;
    }
  }
  uint32_t unused = 0;
  block_sum_max<THREADS>(sum, unused);
  const double mean = static_cast<double>(big) * big * (static_cast<double>(sum) / a.K) + a.eps;
  return static_cast<float>(static_cast<double>(__uint_as_float(top)) / sqrt(mean) / 127.0);
}

// The scale of a row from its sum of squares and the bits of max|t|.
// far: the caller has to take far_scale instead.
__device__ __forceinline__ float scale_of(const NormArgs& a, float sum, uint32_t top, bool& far) {
  far = false;
  if (top >= kInfBits) return __uint_as_float(0x7fc00000u);
  const float A = __uint_as_float(top);
  if (!a.norm || top == 0) return __fdiv_rn(A, 127.f);
  const float mean = __fadd_rn(__fdiv_rn(sum, static_cast<float>(a.K)), a.eps);
  far = !(mean <= FLT_MAX) || mean < 1e-30f;
  return __fdiv_rn(__fmul_rn(A, __frsqrt_rn(mean)), 127.f);
}

// A block for each row, which it reads twice (the second time from L2): any
// row length.
template <class T, int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_loop_kernel(const NormArgs a) {
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    float sum = 0.f;
    uint32_t top = 0;
    for (int c = threadIdx.x * VEC; c < a.K; c += kNormThreads * VEC) {
      float h[VEC], w[VEC];
      load_h<T, VEC>(a, m, c, h);
      load_weight<VEC>(a, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sum += h[e] * h[e];
        top = max(top, abs_bits(h[e] * w[e]));
      }
    }
    block_sum_max<kNormThreads>(sum, top);
    bool far;
    float s = scale_of(a, sum, top, far);
    if (far) s = far_scale<T, VEC, kNormThreads>(a, m, top);
    if (threadIdx.x == 0) a.scale[m] = s;
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
cudaError_t run_norm(const NormArgs& a, cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>(a.M, 148 * 64);
  norm_loop_kernel<T, VEC><<<static_cast<unsigned>(blocks), kNormThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

int norm_rows(const NormArgs& a, int dtype, cudaStream_t stream) {
  const int es = dtype_size(dtype), V = 16 / es;
  const bool vec = a.K % V == 0 && rows16(a.x, a.ldx, es) &&
                   (a.residual == nullptr || rows16(a.residual, a.ldr, es)) &&
                   (a.h_out == nullptr || rows16(a.h_out, a.ldh, es)) &&
                   (a.weight == nullptr || is_aligned(a.weight, 16)) && is_aligned(a.q, V) &&
                   a.ldq % V == 0;
  using B = __nv_bfloat16;
  cudaError_t e;
  if (dtype == DLRM_TABLE_F32)
    e = vec ? run_norm<float, 4>(a, stream) : run_norm<float, 1>(a, stream);
  else
    e = vec ? run_norm<B, 8>(a, stream) : run_norm<B, 1>(a, stream);
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

// y = q * scale: a block walks rows, VEC columns a thread.
template <class T, int VEC>
__global__ void __launch_bounds__(256)
    dequant_kernel(const int8_t* q, int64_t ldq, const float* scale, int M, int K, T* y,
                   int64_t ldy) {
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const float s = __ldg(scale + m);
    for (int c = threadIdx.x * VEC; c < K; c += 256 * VEC) {
      float v[VEC];
      if constexpr (VEC == 1) {
        v[0] = static_cast<float>(q[m * ldq + c]) * s;
      } else {
        const uint2 r = __ldg(reinterpret_cast<const uint2*>(q + m * ldq + c));
        const uint32_t w[2] = {r.x, r.y};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = static_cast<float>(static_cast<int8_t>(w[e / 4] >> (8 * (e % 4)))) * s;
      }
      store_f32<T, VEC>(y + m * ldy + c, v);
    }
  }
}

template <class T>
cudaError_t run_dequant(const int8_t* q, int64_t ldq, const float* scale, int64_t M, int64_t K,
                        T* y, int64_t ldy, cudaStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(M, 148 * 64));
  const bool vec = K % 8 == 0 && is_aligned(q, 8) && ldq % 8 == 0 && rows16(y, ldy, sizeof(T));
  if (vec)
    dequant_kernel<T, 8><<<blocks, 256, 0, stream>>>(q, ldq, scale, static_cast<int>(M),
                                                     static_cast<int>(K), y, ldy);
  else
    dequant_kernel<T, 1><<<blocks, 256, 0, stream>>>(q, ldq, scale, static_cast<int>(M),
                                                     static_cast<int>(K), y, ldy);
  return cudaGetLastError();
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
