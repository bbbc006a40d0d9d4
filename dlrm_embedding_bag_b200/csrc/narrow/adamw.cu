// One AdamW step over many tensors (declared in dlrm_optim.h).
//
// A step reads and writes every element once: 28 bytes an element for f32 with 32-bit
// moments, 16 with 8-bit ones, 10 for bf16 with 8-bit ones. Bound by memory (10^6 x 64 in
// a graph: f32 262 us of 273 by a copy's rate), but with 8-bit moments by instructions (f32
// 166 of 156, bf16 167 of 98; the integer pipe at 58 and 64 %, 0.76 and 0.83 instructions a
// scheduler and cycle). Tensors travel as pointers by value in the launch (up to kMaxTensors
// of them), so a network's dozens of small tensors are one launch and need no copy in front of it.
//
// A warp takes a block of 256 elements, a lane eight neighbours, so that its accesses are
// few and wide (16 bytes of bf16, 8 of codes) and a block's largest moment is one warp
// reduction. Four warps take a chunk of 1024.
// CTAs stay, and chunks are handed out in order by a counter: walking with a fixed
// stride, CTAs drift apart and memory sees a wider and wider window of addresses (10^6 x
// 64 f32 with 32-bit moments 282 us, with 8-bit ones 195; by tickets 261 and 167).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <climits>

#include <cuda_fp16.h>

#include "dlrm_optim.h"
#include "sectors.cuh"
#include "tickets.h"
#include "tokens/common.h"

namespace dlrm {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlock = DLRM_ADAMW_BLOCK;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = kWarps * kBlock;
// Tensors of one launch: 40 bytes each in its arguments, of which 4 KB are room for 96. Few
// take a launch with room for 16, which is sooner made (a call for 12 tensors 9.3 and 7.4 us
// of the host's time).
constexpr int kMaxTensors = 96;
constexpr int kFewTensors = 16;
constexpr int kCtasPerSm = 8;

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

struct StepArgs {
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
template <int ROOM>
struct ListArgs {
  StepArgs step;
  Tensor t[ROOM];
};

// What the whole step shares.
struct Factors {
  float b1, b1c, b2, b2c;  // the decays of the moments and what is left to 1
  float lr, alpha, root;   // alpha = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t)
  float grad_scale;
  uint32_t t, key;         // the step's number, and the key of its random numbers
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

// 8 elements at p.
template <class T, bool ALL>
__device__ __forceinline__ void load8(const T* p, int left, Pair* v) {
  if constexpr (ALL && sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 r = reinterpret_cast<const float4*>(p)[i];
      v[2 * i] = pair(r.x, r.y), v[2 * i + 1] = pair(r.z, r.w);
    }
  } else if constexpr (ALL) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pair(2 * i < left ? static_cast<float>(p[2 * i]) : 0.f,
                  2 * i + 1 < left ? static_cast<float>(p[2 * i + 1]) : 0.f);
  }
}

template <class T, bool ALL>
__device__ __forceinline__ void store8(T* p, int left, const Pair* v) {
  float e[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = parts(v[i]);
    e[2 * i] = f.x, e[2 * i + 1] = f.y;
  }
  if constexpr (ALL) {
#pragma unroll
    for (int i = 0; i < 8; i += 16 / sizeof(T)) store_16_bytes(p + i, e + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = static_cast<T>(e[i]);
  }
}

__device__ __forceinline__ Pair of_halves(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pair(f.x, f.y);
}
// Four codes as numbers without their scale: e4m3, and the roots' unsigned form (4 bits of
// exponent, 4 of mantissa), which is a half-precision number without its sign, the
// exponent's first bit and the mantissa's last six.
__device__ __forceinline__ void first_values(uint32_t c, Pair* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(c >> (16 * i))));
    v[i] = of_halves(h);
  }
}
__device__ __forceinline__ void root_values(uint32_t c, Pair* r) {
  r[0] = of_halves(__byte_perm(c, 0, 0x4140) << 6);
  r[1] = of_halves(__byte_perm(c, 0, 0x4342) << 6);
}

// Numbers become codes by their own bits: times the power of two that brings the format's
// least normal number to that of f32, exponent and upper mantissa are the code (below
// it too: f32's subnormal numbers have even steps as the format's have). Random bits are added
// below the code's last one before the rest is cut off. They are less than a step by
// 2^-16 of one, and the block's largest is above the largest code by 2^-17 of a step at
// most, so no code is left at its upper end.
constexpr float kFirstLower = 0x1p-120f, kRootLower = 0x1p-112f;
// bits + (the low or the high 16 bits of a random word, times UNIT): one dot product of
// halves and bytes, off the pipe of shifts and logic, which is the busiest here.
template <int UNIT>
__device__ __forceinline__ uint32_t plus_low(uint32_t word, uint32_t bits) {
  return __dp2a_lo(word, static_cast<uint32_t>(UNIT), bits);
}
template <int UNIT>
__device__ __forceinline__ uint32_t plus_high(uint32_t word, uint32_t bits) {
  return __dp2a_lo(word, static_cast<uint32_t>(UNIT) << 8, bits);
}
// The upper bytes of four words.
__device__ __forceinline__ uint32_t upper_bytes(const uint32_t (&t)[4]) {
  return __byte_perm(__byte_perm(t[0], t[1], 0x0073), __byte_perm(t[2], t[3], 0x0073), 0x5410);
}

// The function units' root and reciprocal. The root serves what near_root does not: zero, subnormal
// numbers and what is not finite. The reciprocal is within a last place, and a step needs no more
// of its own size.
__device__ __forceinline__ float root_of(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The second moment's root, which becomes a code, is the nearest f32 from moments of 2^-108 on (all
// of 4 * 10^6 were): one step of Newton's method, r + (x - r^2) / (2 r), from r = x y, where y is
// about 1 / sqrt(x). Below 2^-108 what r^2 leaves of x ends at 2^-149, and the root is within a last
// place of it (at 2^-126 one of 13 is another number than the nearest). 0 below 2^-126, NaN of
// what is not finite.
__device__ __forceinline__ float inverse_root(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r > 0x1.8p63f ? 0.f : r;
}
__device__ __forceinline__ Pair near_root(Pair x) {
  const float2 f = parts(x);
  const Pair y = pair(inverse_root(f.x), inverse_root(f.y)), r = mul(x, y);
  return fma(fma(mul(r, both(-1.f)), r, x), mul(y, both(0.5f)), r);
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Towards bf16 by chance: what a cut after the upper half makes of it goes up with the
// probability of what is left over. (An infinity has nothing to carry; NaN is not given.)
__device__ __forceinline__ float by_chance(float x, uint32_t word) {
  return __uint_as_float(plus_high<1>(word * 0x3C6EF373u, __float_as_uint(x)));
}
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// One block of 256 elements of a tensor by one warp; `left` elements of it are there.
template <int BITS, class P, class G, bool ALL>
__device__ __forceinline__ void step_block(const StepArgs& a, const Factors& f, const Tensor& t,
                                           int64_t e0, int left) {
  const int lane = threadIdx.x & 31;
  const int q = lane * 8;  // the lane's first place in the block
  const uint32_t block = t.block0 + static_cast<uint32_t>(e0 / kBlock);
  const int64_t at = static_cast<int64_t>(block) * kBlock;
  P* param = static_cast<P*>(t.param) + e0;
  const G* grad = static_cast<const G*>(t.grad) + e0;
  const bool whole = sizeof(P) == 2 && a.master != nullptr;

  Pair p[4], g[4], m[4], v[4];
  uint32_t mc[2], vc[2];
  float ms = 1.f, vs = 1.f;  // the scales of what was read
  load8<G, ALL>(grad + q, left - q, g);
  if (whole)
    load8<float, true>(a.master + at + q, 8, p);
  else
    load8<P, ALL>(param + q, left - q, p);
  if constexpr (BITS == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.m) + at + q);
    const uint2 y = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + at + q);
    mc[0] = x.x, mc[1] = x.y, vc[0] = y.x, vc[1] = y.y;
  } else {
    load8<float, true>(static_cast<const float*>(a.m) + at + q, 8, m);
    load8<float, true>(static_cast<const float*>(a.v) + at + q, 8, v);
  }
  // a random word for each element, while those are on their way
  uint32_t word[8];
  if constexpr (BITS == 8 || sizeof(P) == 2) {
    const uint32_t base = mixed(f.key ^ block) + static_cast<uint32_t>(q) * 0x9E3779B9u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      word[i] = mixed(base + static_cast<uint32_t>(i) * 0x9E3779B9u);
  }
  if constexpr (BITS == 8) {
    ms = a.m_scale[block];
    vs = a.v_scale[block];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      first_values(mc[h], m + 2 * h);
      root_values(vc[h], v + 2 * h);
    }
  }
  // Moments round after every product and sum, as elementary operations do: where a code
  // goes up or down then hangs on the formula alone (and on the root below), not on what was fused.
  // (10^6 x 64 with 8-bit moments, fused and with a root off by a last place: f32 155 us, bf16 148, so
  // 166 and 167; that sent 1.5 of 10^6 codes the other way, and in the next step some weights with them.)
  const Pair b1 = both(f.b1), b1c = both(f.b1c), b2 = both(f.b2), b2c = both(f.b2c);
  const Pair scale = both(f.grad_scale), keep = both(__fmaf_rn(-f.lr, t.decay, 1.f));
  const Pair alpha = both(-f.alpha), root = both(f.root), eps = both(a.eps);
  Pair r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Pair x = mul(g[i], scale);
    if constexpr (BITS == 8) {
      m[i] = mul(m[i], both(ms));
      v[i] = mul(v[i], both(vs));
      v[i] = mul(v[i], v[i]);
    }
    m[i] = add(mul(m[i], b1), mul(x, b1c));
    v[i] = add(mul(v[i], b2), mul(mul(x, x), b2c));
    if constexpr (BITS == 8) {
      r[i] = near_root(v[i]);
    } else {
      const float2 w = parts(v[i]), y = parts(near_root(v[i]));
      r[i] = pair(w.x >= FLT_MIN && w.x <= FLT_MAX ? y.x : root_of(w.x),
                  w.y >= FLT_MIN && w.y <= FLT_MAX ? y.y : root_of(w.y));
    }
  }
  float vf = 0.f;  // the lane's largest root, NaN if one is
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = parts(r[i]);
      vf = max_abs(vf, y.x, y.y);
    }
    if (vf != vf) {  // an infinity stays one: a square may leave f32 where its gradient does not
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 w = parts(v[i]);
        r[i] = pair(root_of(w.x), root_of(w.y));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 d = parts(fma(r[i], root, eps));
    p[i] = fma(mul(m[i], pair(reciprocal(d.x), reciprocal(d.y))), alpha, mul(p[i], keep));
  }
  if constexpr (!ALL) {
    // what lies behind the tensor's end stays zero, whatever the factors are
    vf = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = q + 2 * i;
      const float2 pe = parts(p[i]), me = parts(m[i]), ve = parts(v[i]), re = parts(r[i]);
      const bool lo = e < left, hi = e + 1 < left;
      p[i] = pair(lo ? pe.x : 0.f, hi ? pe.y : 0.f);
      m[i] = pair(lo ? me.x : 0.f, hi ? me.y : 0.f);
      v[i] = pair(lo ? ve.x : 0.f, hi ? ve.y : 0.f);
      r[i] = pair(lo ? re.x : 0.f, hi ? re.y : 0.f);
      vf = max_abs(vf, lo ? re.x : 0.f, hi ? re.y : 0.f);
    }
  }
  if constexpr (BITS == 8) {
    float mf = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = parts(m[i]);
      mf = max_abs(mf, x.x, x.y);
    }
    // (of numbers that are not negative the bits' order is theirs, and NaN is above all)
    const uint32_t mtop = __reduce_max_sync(kFull, __float_as_uint(mf));
    const uint32_t vtop = __reduce_max_sync(kFull, __float_as_uint(vf));
    mf = __uint_as_float(mtop), vf = __uint_as_float(vtop);
    const bool mbad = mtop >= 0x7f800000u, vbad = vtop >= 0x7f800000u;
    const bool live = mf >= 448.f * 0x1p-126f && !mbad;
    const Pair minv = both(live ? __fmul_rn(__frcp_rn(mf), 448.f) : 0.f), mlow = both(kFirstLower);
    const Pair vinv = both(vtop != 0 && !vbad ? __fmul_rn(__frcp_rn(vf), 1.9375f) : 0.f), vlow = both(kRootLower);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[4], z[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 mx = parts(mul(mul(m[2 * h + i], minv), mlow));
        const float2 rx = parts(mul(mul(r[2 * h + i], vinv), vlow));
        x[2 * i] = __float_as_uint(mx.x), x[2 * i + 1] = __float_as_uint(mx.y);
        z[2 * i] = __float_as_uint(rx.x), z[2 * i + 1] = __float_as_uint(rx.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the code to the top of its word; the sign in front of the first moment's seven bits
        const uint32_t w = word[4 * h + i];
        x[i] = (plus_low<16>(w, x[i]) * 16u & 0x7fffffffu) | (x[i] & 0x80000000u);
        z[i] = plus_high<8>(w, z[i]) * 32u;
      }
      mc[h] = upper_bytes(x);
      vc[h] = upper_bytes(z);
      // A root that is not zero stays so: a look at each only where one of four codes is zero.
      if ((vc[h] - 0x01010101u) & ~vc[h] & 0x80808080u) {
        const float2 y = parts(r[2 * h]), z = parts(r[2 * h + 1]);
        if (y.x > 0.f && (vc[h] & 0xffu) == 0) vc[h] |= 1u;
        if (y.y > 0.f && (vc[h] & 0xff00u) == 0) vc[h] |= 1u << 8;
        if (z.x > 0.f && (vc[h] & 0xff0000u) == 0) vc[h] |= 1u << 16;
        if (z.y > 0.f && (vc[h] & 0xff000000u) == 0) vc[h] |= 1u << 24;
      }
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + at + q) =
        live ? make_uint2(mc[0], mc[1]) : make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + at + q) =
        vbad ? make_uint2(0u, 0u) : make_uint2(vc[0], vc[1]);
    if (lane == 0) {
      const float nan = __uint_as_float(0x7fc00000u);
      a.m_scale[block] = mbad ? nan : live ? mf * (1.f / 448.f) : 0.f;
      a.v_scale[block] = vbad ? nan : vf * (1.f / 1.9375f);
    }
  } else {
    store8<float, true>(static_cast<float*>(a.m) + at + q, 8, m);
    store8<float, true>(static_cast<float*>(a.v) + at + q, 8, v);
  }
  if (whole) {
    store8<float, true>(a.master + at + q, 8, p);
  } else if constexpr (sizeof(P) == 2) {
    uint32_t b[4];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = parts(p[i]);
      b[i] = upper_halves(by_chance(y.x, word[2 * i]), by_chance(y.y, word[2 * i + 1]));
      top = max_abs(top, y.x, y.y);
    }
    if (top != top) {  // with a NaN among them: by the conversion that keeps it
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = parts(p[i]);
        b[i] = upper_halves(y.x != y.x ? y.x : by_chance(y.x, word[2 * i]),
                            y.y != y.y ? y.y : by_chance(y.y, word[2 * i + 1]));
      }
    }
    if constexpr (ALL) {
      *reinterpret_cast<uint4*>(param + q) = make_uint4(b[0], b[1], b[2], b[3]);
    } else {
      uint16_t* at_p = reinterpret_cast<uint16_t*>(param + q);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (q + i < left) at_p[i] = static_cast<uint16_t>(b[i / 2] >> (16 * (i % 2)));
    }
    return;
  }
  store8<P, ALL>(param + q, left - q, p);
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

// The word that chunks are counted in. (Taken from the arguments at each use: its address in two
// registers for the whole walk cost 1 %.)
__device__ __forceinline__ uint32_t* counter(const StepArgs& a) {
  return reinterpret_cast<uint32_t*>(a.step + 1);
}

template <int BITS, int ROOM>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    adamw_kernel(const __grid_constant__ ListArgs<ROOM> args) {
  const StepArgs& a = args.step;
  __shared__ Factors shared;
  __shared__ int next[2];
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) atomicMax(counter(a), kDrawing);
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
    shared.t = t;
    shared.key = mixed(mixed(a.seed + 0x9E3779B9u) ^ t);
    // (Most find it raised by now: with one maximum for each of 577 CTAs 5.8 us, so 5.6.)
    const uint32_t seen = *static_cast<volatile uint32_t*>(counter(a));
    if (!raised(seen)) atomicCAS(counter(a), seen, kDrawing);
    __threadfence();  // the count is read before this CTA draws a ticket
  }
  __syncthreads();
  const Factors f = shared;
  const int warp = threadIdx.x >> 5;
  // Chunks are handed out in order, by tickets that a CTA draws while it works on the chunk
  // before (tickets.h).
  int ti = 0;
  for (int c = blockIdx.x, turn = 0;; turn ^= 1) {
    uint32_t drawn = 0;
    if (threadIdx.x == 0) drawn = atomicAdd(counter(a), 1u);
    if (c < a.chunks) {
      // the last tensor that starts at c or before it: near the last one, but for the first
      // chunk
      if (c == static_cast<int>(blockIdx.x)) {
        for (int hi = a.n; hi - ti > 1;) {
          const int mid = (ti + hi) >> 1;
          if (args.t[mid].first <= c)
            ti = mid;
          else
            hi = mid;
        }
      } else {
        while (ti + 1 < a.n && args.t[ti + 1].first <= c) ++ti;
      }
      const Tensor& t = args.t[ti];
      const int64_t e0 = static_cast<int64_t>(c - t.first) * kChunk + warp * kBlock;
      switch (t.flags & (kParamBf16 | kGradBf16)) {
        case 0: step_warp<BITS, float, float>(a, f, t, e0); break;
        case kParamBf16: step_warp<BITS, __nv_bfloat16, float>(a, f, t, e0); break;
        case kGradBf16: step_warp<BITS, float, __nv_bfloat16>(a, f, t, e0); break;
        default: step_warp<BITS, __nv_bfloat16, __nv_bfloat16>(a, f, t, e0); break;
      }
    }
    if (threadIdx.x == 0) {
      next[turn] = next_chunk(drawn, a.chunks, static_cast<int>(gridDim.x));
      if (last_ticket(drawn, a.chunks)) {
        // every CTA has read the count and drawn its last ticket
        *counter(a) = 0;
        if (a.last) a.step[0] = static_cast<int32_t>(f.t);
      }
    }
    __syncthreads();
    c = next[turn];
    if (c >= a.chunks) break;
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
  const Pair mp = both(ms), vp = both(vs);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    Pair x[2], y[2];
    first_values(mw[i], x);
    root_values(vw[i], y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 first = parts(mul(x[k], mp));
      y[k] = mul(y[k], vp);
      const float2 second = parts(mul(y[k], y[k]));
      mf[4 * i + 2 * k] = first.x, mf[4 * i + 2 * k + 1] = first.y;
      vf[4 * i + 2 * k] = second.x, vf[4 * i + 2 * k + 1] = second.y;
    }
  }
  store_sectors(m_out + at, mf);
  store_sectors(v_out + at, vf);
}

template <int ROOM>
cudaError_t launch_step(int bits, const StepArgs& a, const Tensor* t, int sms, cudaStream_t s) {
  ListArgs<ROOM> args;
  args.step = a;
  std::copy(t, t + a.n, args.t);
  const int grid = std::max(1, std::min(a.chunks, sms * kCtasPerSm));
  return launch(bits == 8 ? &adamw_kernel<8, ROOM> : &adamw_kernel<32, ROOM>,
                dim3(static_cast<unsigned>(grid)), kThreads, 0, false, s, args);
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
  if (!(static_cast<float>(eps) >= FLT_MIN) || !std::isfinite(static_cast<float>(eps)))
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
    if (blocks >= (int64_t{1} << 32) || chunks > int64_t{kMostTickets}) return DLRM_ERR_SHAPE;
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
  const auto s = static_cast<cudaStream_t>(stream);
  StepArgs a = {};
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
  int64_t i = 0, block = 0;
  do {
    Tensor list[kMaxTensors];
    a.n = a.chunks = 0;
    for (; i < n && a.n < kMaxTensors; ++i) {
      if (counts[i] == 0) continue;
      Tensor& t = list[a.n++];
      t.param = params[i];
      t.grad = grads[i];
      t.count = counts[i];
      t.block0 = static_cast<uint32_t>(block);
      t.first = a.chunks;
      t.decay = decays != nullptr ? decays[i] : 0.f;
      t.flags = (param_dtypes[i] == DLRM_TABLE_BF16 ? kParamBf16 : 0) |
                (grad_dtypes[i] == DLRM_TABLE_BF16 ? kGradBf16 : 0) |
                (is_aligned(params[i], 16) && is_aligned(grads[i], 16) ? kAligned : 0);
      block += (counts[i] + kBlock - 1) / kBlock;
      a.chunks += static_cast<int>((counts[i] + kChunk - 1) / kChunk);
    }
    while (i < n && counts[i] == 0) ++i;
    a.last = i >= n;
    const cudaError_t e = a.n <= kFewTensors ? launch_step<kFewTensors>(bits, a, list, sms, s)
                                             : launch_step<kMaxTensors>(bits, a, list, sms, s);
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
      !is_aligned(v_scale, 4) || !is_aligned(m_out, 32) || !is_aligned(v_out, 32))
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
