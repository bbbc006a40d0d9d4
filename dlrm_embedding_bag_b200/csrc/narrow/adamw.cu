// One AdamW step over many tensors (declared in dlrm_optim.h).
//
// A step reads and writes every element once and computes some 40 to 70
// instructions on it, so it is bound by memory: 28 bytes an element for f32 with
// 32-bit moments, 16 with 8-bit ones, 10 for bf16 with 8-bit ones. Tensors travel as pointers by
// value in the launch (up to kMaxTensors of them), so a network's dozens of small
// tensors are one launch and need no copy in front of it.
//
// A warp takes a block of 256 elements, a lane four neighbours in either half, so
// that every access of a warp is whole lines (512 bytes of f32, 128 of codes)
// and a block's largest moment is one warp reduction. Eight warps take a chunk of
// 2048; CTAs stay and walk over the chunks.
#include <cmath>
#include <climits>

#include <cuda_fp16.h>

#include "dlrm_optim.h"
#include "tokens/common.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlock = DLRM_ADAMW_BLOCK;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = kWarps * kBlock;
constexpr int kMaxTensors = 96;  // of one launch: their 40 bytes each fit the classic 4 KB of arguments
constexpr int kCtasPerSm = 4;

enum TensorFlags { kParamBf16 = 1, kGradBf16 = 2, kAligned = 4 };

struct Tensor {
  void* param;
  const void* grad;
  int64_t count;
  uint32_t block0;  // its first block of the arena
  int first;        // its first chunk of this launch
  float decay;
  int flags;
};

struct alignas(16) StepArgs {
  Tensor t[kMaxTensors];
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int32_t* step;
  const float* lr_dev;
  const float* grad_scale;
  double lr, beta1, beta2;
  float eps;
  uint32_t seed;
  int n, chunks;
  int last;  // whether this launch ends the step
};

// What the whole step shares.
struct Factors {
  float b1, b1c, b2, b2c;  // the decays of the moments and what is left to 1
  float lr, alpha, root;   // alpha = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t)
  float grad_scale;
  uint32_t key;  // of this step's random numbers
};

// b^t by squaring, in 64 bits: a few of their roundings off.
__device__ double power(double b, uint32_t t) {
  double r = 1.0;
  for (; t != 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// 32 bits that look random from 32 that do not: products with odd numbers (the
// fractions of the roots of 2 and 3) spread the low bits upwards, the shifts the high
// ones down. Two rounds: every input bit reaches every output bit.
__device__ __forceinline__ uint32_t mixed(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// 4 elements at p.
template <class T, bool ALL>
__device__ __forceinline__ void load4(const T* p, int left, float* v) {
  if constexpr (ALL) {
    if constexpr (sizeof(T) == 4) {
      const float4 r = *reinterpret_cast<const float4*>(p);
      v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    } else {
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
      v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? static_cast<float>(p[i]) : 0.f;
  }
}

template <class T, bool ALL>
__device__ __forceinline__ void store4(T* p, int left, const float* v) {
  if constexpr (ALL) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) {
        if constexpr (sizeof(T) == 4)
          p[i] = v[i];
        else
          p[i] = __float2bfloat16_rn(v[i]);
      }
  }
}

// Four codes as values: e4m3, and the roots' unsigned form (4 bits of exponent, 4 of
// mantissa): its bits in an f32's exponent and mantissa (where a code without exponent is a
// subnormal number, as the format has it), whose bias 2^112 corrects.
__device__ __forceinline__ void first_values(uint32_t c, float scale, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(c >> (16 * i))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}
__device__ __forceinline__ void root_values(uint32_t c, float scale, float* r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = i < 3 ? c << (19 - 8 * i) : c >> 5;
    r[i] = __uint_as_float(at & (0xffu << 19)) * 0x1p112f * scale;
  }
}

// x >= 0 as a code of FRAC mantissa bits: times the power of two that brings the format's
// least normal number to that of f32, its exponent and upper mantissa bits are the code (below
// it too: f32's subnormal numbers have even steps as the format's have), rounded down
// after `chance`, random bits below the code's last one, was added.
template <int FRAC, int LEAST, int TOP>
__device__ __forceinline__ uint32_t code_of(float x, uint32_t chance) {
  constexpr float kLower = LEAST == -6 ? 0x1p-120f : 0x1p-112f;
  static_assert(LEAST == -6 || LEAST == -14, "2^(-126 - LEAST)");
  return min((__float_as_uint(x * kLower) + chance) >> (23 - FRAC), static_cast<uint32_t>(TOP));
}

// Root and quotient from the function units: within two last places, where an element's
// step needs no more than that of its own size.
__device__ __forceinline__ float root_of(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float quotient(float a, float b) {
  float r;
  asm("div.approx.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// bf16 by chance: up with the probability of what is left over. Not a number and infinite
// stay so.
__device__ __forceinline__ float by_chance(float x, uint32_t chance) {
  const uint32_t b = __float_as_uint(x);
  if ((b & 0x7f800000u) == 0x7f800000u) return x;
  return __uint_as_float((b + chance) & 0xffff0000u);
}

// One block of 256 elements of a tensor by one warp; `left` elements of it are there.
template <int BITS, class P, class G, bool ALL>
__device__ __forceinline__ void step_block(const StepArgs& a, const Factors& f, const Tensor& t,
                                           int64_t e0, int left) {
  const int lane = threadIdx.x & 31;
  const int q[2] = {lane * 4, 128 + lane * 4};  // the lane's places in the block
  const uint32_t block = t.block0 + static_cast<uint32_t>(e0 / kBlock);
  const int64_t at = static_cast<int64_t>(block) * kBlock;
  P* param = static_cast<P*>(t.param) + e0;
  const G* grad = static_cast<const G*>(t.grad) + e0;
  const bool whole = sizeof(P) == 2 && a.master != nullptr;

  float p[8], g[8], m[8], v[8];
  uint32_t mc[2], vc[2];
  float ms = 0.f, vs = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load4<G, ALL>(grad + q[h], left - q[h], g + 4 * h);
    if (whole)
      load4<float, true>(a.master + at + q[h], 4, p + 4 * h);
    else
      load4<P, ALL>(param + q[h], left - q[h], p + 4 * h);
    if constexpr (BITS == 8) {
      mc[h] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.m) + at + q[h]);
      vc[h] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v) + at + q[h]);
    } else {
      load4<float, true>(static_cast<const float*>(a.m) + at + q[h], 4, m + 4 * h);
      load4<float, true>(static_cast<const float*>(a.v) + at + q[h], 4, v + 4 * h);
    }
  }
  if constexpr (BITS == 8) {
    ms = a.m_scale[block];
    vs = a.v_scale[block];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      first_values(mc[h], ms, m + 4 * h);
      root_values(vc[h], vs, v + 4 * h);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] *= v[4 * h + i];
    }
  }
  const float keep = __fmaf_rn(-f.lr, t.decay, 1.f);
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = g[i] * f.grad_scale;
    m[i] = __fmaf_rn(m[i], f.b1, x * f.b1c);
    v[i] = __fmaf_rn(v[i], f.b2, x * x * f.b2c);
    r[i] = root_of(v[i]);
    p[i] = __fmaf_rn(-f.alpha, quotient(m[i], __fmaf_rn(r[i], f.root, a.eps)), p[i] * keep);
  }
  // a random word for each element
  uint32_t word[8];
  if constexpr (BITS == 8 || sizeof(P) == 2) {
    const uint32_t base = mixed(f.key ^ block);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      word[i] = mixed(base + static_cast<uint32_t>(q[i / 4] + i % 4) * 0x9E3779B9u);
  }
  if constexpr (BITS == 8) {
    // what lies behind the tensor's end stays zero: its gradient was read as zero
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mtop = max(mtop, __float_as_uint(fabsf(m[i])));
      vtop = max(vtop, __float_as_uint(fabsf(r[i])));
    }
    mtop = __reduce_max_sync(kFull, mtop);
    vtop = __reduce_max_sync(kFull, vtop);
    const bool mbad = mtop >= 0x7f800000u, vbad = vtop >= 0x7f800000u;
    float mscale = __fdiv_rn(__uint_as_float(mtop), 448.f);
    const bool live = mscale >= 0x1p-126f && !mbad;
    const float minv = live ? __fdiv_rn(448.f, __uint_as_float(mtop)) : 0.f;
    if (!live) mscale = 0.f;
    const float vscale = __fdiv_rn(__uint_as_float(vtop), 1.9375f);
    const float vinv = vtop != 0 && !vbad ? __fdiv_rn(1.9375f, __uint_as_float(vtop)) : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[4], d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * h + i;
        c[i] = code_of<3, -6, 126>(fabsf(m[k]) * minv, (word[k] & 0xffffu) << 4);
        d[i] = code_of<4, -14, 255>(r[k] * vinv, (word[k] >> 16) << 3);
        d[i] = max(d[i], min(__float_as_uint(r[k]), 1u));  // what is not zero stays so
      }
      const uint32_t signs =
          __byte_perm(__byte_perm(__float_as_uint(m[4 * h]), __float_as_uint(m[4 * h + 1]), 0x0073),
                      __byte_perm(__float_as_uint(m[4 * h + 2]), __float_as_uint(m[4 * h + 3]), 0x0073),
                      0x5410);
      mc[h] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24 | (signs & 0x80808080u);
      vc[h] = d[0] | d[1] << 8 | d[2] << 16 | d[3] << 24;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + at + q[h]) = live ? mc[h] : 0u;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + at + q[h]) = vbad ? 0u : vc[h];
    }
    if (lane == 0) {
      const float nan = __uint_as_float(0x7fc00000u);
      a.m_scale[block] = mbad ? nan : mscale;
      a.v_scale[block] = vbad ? nan : vscale;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      store4<float, true>(static_cast<float*>(a.m) + at + q[h], 4, m + 4 * h);
      store4<float, true>(static_cast<float*>(a.v) + at + q[h], 4, v + 4 * h);
    }
  }
  if (whole) {
#pragma unroll
    for (int h = 0; h < 2; ++h) store4<float, true>(a.master + at + q[h], 4, p + 4 * h);
  } else if constexpr (sizeof(P) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = by_chance(p[i], (word[i] * 0x3C6EF373u) >> 16);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) store4<P, ALL>(param + q[h], left - q[h], p + 4 * h);
}

template <int BITS, class P, class G>
__device__ __forceinline__ void step_warp(const StepArgs& a, const Factors& f, const Tensor& t,
                                          int64_t e0) {
  const int64_t left = t.count - e0;
  if (left <= 0) return;
  if (left >= kBlock && (t.flags & kAligned))
    step_block<BITS, P, G, true>(a, f, t, e0, kBlock);
  else
    step_block<BITS, P, G, false>(a, f, t, e0, left < kBlock ? static_cast<int>(left) : kBlock);
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    adamw_kernel(const __grid_constant__ StepArgs a) {
  __shared__ Factors shared;
  if (threadIdx.x == 0) {
    const uint32_t t = static_cast<uint32_t>(a.step[0]) + 1u;
    const double lr = a.lr_dev != nullptr ? static_cast<double>(*a.lr_dev) : a.lr;
    shared.b1 = static_cast<float>(a.beta1);
    shared.b1c = static_cast<float>(1.0 - a.beta1);
    shared.b2 = static_cast<float>(a.beta2);
    shared.b2c = static_cast<float>(1.0 - a.beta2);
    shared.lr = static_cast<float>(lr);
    shared.alpha = static_cast<float>(lr / (1.0 - power(a.beta1, t)));
    shared.root = static_cast<float>(1.0 / sqrt(1.0 - power(a.beta2, t)));
    shared.grad_scale = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
    shared.key = mixed(mixed(a.seed + 0x9E3779B9u) ^ t);
    if (a.last) {
      // the last CTA to have read the count writes the next one
      __threadfence();
      if (atomicAdd(a.step + 1, 1) == static_cast<int>(gridDim.x) - 1) {
        a.step[1] = 0;
        a.step[0] = static_cast<int32_t>(t);
      }
    }
  }
  __syncthreads();
  const Factors f = shared;
  const int warp = threadIdx.x >> 5;
  int ti = 0;
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    // the last tensor that starts at c or before it
    int hi = a.n;
    while (hi - ti > 1) {
      const int mid = (ti + hi) >> 1;
      if (a.t[mid].first <= c)
        ti = mid;
      else
        hi = mid;
    }
    const Tensor& t = a.t[ti];
    const int64_t e0 = static_cast<int64_t>(c - t.first) * kChunk + warp * kBlock;
    switch (t.flags & (kParamBf16 | kGradBf16)) {
      case 0: step_warp<BITS, float, float>(a, f, t, e0); break;
      case kParamBf16: step_warp<BITS, __nv_bfloat16, float>(a, f, t, e0); break;
      case kGradBf16: step_warp<BITS, float, __nv_bfloat16>(a, f, t, e0); break;
      default: step_warp<BITS, __nv_bfloat16, __nv_bfloat16>(a, f, t, e0); break;
    }
  }
}

// 8-bit moments as values: 16 elements a thread.
template <class T>
__global__ void __launch_bounds__(256)
    moments_kernel(int64_t count, const uint8_t* m, const uint8_t* v, const float* m_scale,
                   const float* v_scale, T* m_out, T* v_out) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 16;
  if (at >= count) return;
  const uint4 mc = *reinterpret_cast<const uint4*>(m + at);
  const uint4 vc = *reinterpret_cast<const uint4*>(v + at);
  const float ms = m_scale[at / kBlock], vs = v_scale[at / kBlock];
  const uint32_t mw[4] = {mc.x, mc.y, mc.z, mc.w}, vw[4] = {vc.x, vc.y, vc.z, vc.w};
  float mf[16], vf[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    first_values(mw[i], ms, mf + 4 * i);
    root_values(vw[i], vs, vf + 4 * i);
#pragma unroll
    for (int k = 0; k < 4; ++k) vf[4 * i + k] *= vf[4 * i + k];
  }
  constexpr int V = kVecOf<T>;
#pragma unroll
  for (int i = 0; i < 16; i += V) {
    store_f32<T, V>(m_out + at + i, *reinterpret_cast<const float(*)[V]>(mf + i));
    store_f32<T, V>(v_out + at + i, *reinterpret_cast<const float(*)[V]>(vf + i));
  }
}

}  // namespace
}  // namespace dlrm

extern "C" {

int dlrm_adamw_step(int64_t n, void* const* params, const void* const* grads,
                    const int64_t* counts, const int32_t* param_dtypes,
                    const int32_t* grad_dtypes, const float* decays, int bits, void* m, void* v,
                    float* m_scale, float* v_scale, float* master, int32_t* step, double lr,
                    const float* lr_dev, double beta1, double beta2, double eps,
                    const float* grad_scale_dev, uint32_t seed, dlrm_stream_t stream) {
  using namespace dlrm;
  if (n < 0 || n > INT_MAX) return DLRM_ERR_SHAPE;
  if (bits != 8 && bits != 32) return DLRM_ERR_ARG;
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1)) return DLRM_ERR_ARG;
  if (!(static_cast<float>(eps) > 0.f) || !std::isfinite(static_cast<float>(eps)))
    return DLRM_ERR_ARG;
  if (lr_dev == nullptr && !std::isfinite(lr)) return DLRM_ERR_ARG;
  if (step == nullptr) return DLRM_ERR_NULL;
  if (!is_aligned(step, 4) || !is_aligned(lr_dev, 4) || !is_aligned(grad_scale_dev, 4))
    return DLRM_ERR_ALIGN;
  if (n > 0 && (params == nullptr || grads == nullptr || counts == nullptr ||
                param_dtypes == nullptr || grad_dtypes == nullptr))
    return DLRM_ERR_NULL;
  int64_t blocks = 0, chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (counts[i] < 0 || counts[i] >= (int64_t{1} << 40)) return DLRM_ERR_SHAPE;
    blocks += (counts[i] + kBlock - 1) / kBlock;
    chunks += (counts[i] + kChunk - 1) / kChunk;
    if (blocks >= (int64_t{1} << 32) || chunks >= INT_MAX) return DLRM_ERR_SHAPE;
    if (!known_dtype(param_dtypes[i]) || !known_dtype(grad_dtypes[i])) return DLRM_ERR_ARG;
    if (decays != nullptr && !std::isfinite(decays[i])) return DLRM_ERR_ARG;
    if (counts[i] == 0) continue;
    if (params[i] == nullptr || grads[i] == nullptr) return DLRM_ERR_NULL;
    if (!is_aligned(params[i], dtype_size(param_dtypes[i])) ||
        !is_aligned(grads[i], dtype_size(grad_dtypes[i])))
      return DLRM_ERR_ALIGN;
  }
  if (blocks > 0) {
    if (m == nullptr || v == nullptr) return DLRM_ERR_NULL;
    if (bits == 8 && (m_scale == nullptr || v_scale == nullptr)) return DLRM_ERR_NULL;
    if (!is_aligned(m, 16) || !is_aligned(v, 16) || !is_aligned(m_scale, 16) ||
        !is_aligned(v_scale, 16) || !is_aligned(master, 16))
      return DLRM_ERR_ALIGN;
  }
  const int sms = sm_count_current();
  if (sms == 0) return DLRM_ERR_CUDA;
  auto* kernel = bits == 8 ? &adamw_kernel<8> : &adamw_kernel<32>;
  int64_t i = 0, block = 0;
  do {
    StepArgs a;
    a.n = 0;
    int64_t c = 0;
    for (; i < n && a.n < kMaxTensors; ++i) {
      if (counts[i] == 0) continue;
      Tensor& t = a.t[a.n++];
      t.param = params[i];
      t.grad = grads[i];
      t.count = counts[i];
      t.block0 = static_cast<uint32_t>(block);
      t.first = static_cast<int>(c);
      t.decay = decays != nullptr ? decays[i] : 0.f;
      t.flags = (param_dtypes[i] == DLRM_TABLE_BF16 ? kParamBf16 : 0) |
                (grad_dtypes[i] == DLRM_TABLE_BF16 ? kGradBf16 : 0) |
                (is_aligned(params[i], 16) && is_aligned(grads[i], 16) ? kAligned : 0);
      block += (counts[i] + kBlock - 1) / kBlock;
      c += (counts[i] + kChunk - 1) / kChunk;
    }
    while (i < n && counts[i] == 0) ++i;
    a.m = m;
    a.v = v;
    a.m_scale = m_scale;
    a.v_scale = v_scale;
    a.master = master;
    a.step = step;
    a.lr_dev = lr_dev;
    a.grad_scale = grad_scale_dev;
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = static_cast<float>(eps);
    a.seed = seed;
    a.chunks = static_cast<int>(c);
    a.last = i >= n;
    const int64_t most = static_cast<int64_t>(sms) * kCtasPerSm;
    const int grid = static_cast<int>(c < 1 ? 1 : c < most ? c : most);
    const cudaError_t e = launch(kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, false,
                                 static_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return cuda_fail(e);
    note_launch();
  } while (i < n);
  return DLRM_OK;
}

int dlrm_adamw_moments(int64_t count, const void* m, const void* v, const float* m_scale,
                       const float* v_scale, void* m_out, void* v_out, int dtype,
                       dlrm_stream_t stream) {
  using namespace dlrm;
  if (count < 0 || count % kBlock != 0 || count >= (int64_t{1} << 40)) return DLRM_ERR_SHAPE;
  if (!known_dtype(dtype)) return DLRM_ERR_ARG;
  if (count == 0) return DLRM_OK;
  if (m == nullptr || v == nullptr || m_scale == nullptr || v_scale == nullptr ||
      m_out == nullptr || v_out == nullptr)
    return DLRM_ERR_NULL;
  if (!is_aligned(m, 16) || !is_aligned(v, 16) || !is_aligned(m_scale, 4) ||
      !is_aligned(v_scale, 4) || !is_aligned(m_out, 16) || !is_aligned(v_out, 16))
    return DLRM_ERR_ALIGN;
  const dim3 grid(static_cast<unsigned>((count / 16 + 255) / 256));
  const auto* mb = static_cast<const uint8_t*>(m);
  const auto* vb = static_cast<const uint8_t*>(v);
  const auto s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dtype == DLRM_TABLE_F32
          ? launch(&moments_kernel<float>, grid, 256, 0, false, s, count, mb, vb, m_scale, v_scale,
                   static_cast<float*>(m_out), static_cast<float*>(v_out))
          : launch(&moments_kernel<__nv_bfloat16>, grid, 256, 0, false, s, count, mb, vb, m_scale,
                   v_scale, static_cast<__nv_bfloat16*>(m_out), static_cast<__nv_bfloat16*>(v_out));
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

}  // extern "C"
