// The layer on 8-bit integers (declared in dlrm_int8.h):
// y[m][n] = act(x_scale[m] * w_scale[n] * sum_k x[m][k] w[n][k] + bias[n]).
#include <algorithm>
#include <climits>

#include "common.h"
#include "dlrm_int8.h"

namespace dlrm {
namespace {

struct LinArgs {
  const int8_t* x;
  const int8_t* w;
  const float* x_scale;
  const float* w_scale;
  const float* bias;
  void* y;
  int64_t ldx, ldw, ldy;
  int M, N, K;
  int act, y_bf16;
  int32_t* status;
};

__device__ __forceinline__ float activate(float x, int act) {
  if (act == DLRM_ACT_RELU) return x > 0.f ? x : (x != x ? x : 0.f);
  if (act == DLRM_ACT_SIGMOID) return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x)));
  return x;
}

__device__ __forceinline__ float finish(const LinArgs& a, int acc, float xs, float ws, float b) {
  return activate(__fadd_rn(static_cast<float>(acc) * xs * ws, b), a.act);
}

// 64 x 64 outputs a block, 4 x 4 a thread, four products an instruction.
constexpr int kTile = 64, kStepK = 64;

// 16 bytes of row r at column k, zero past the row's K columns.
__device__ __forceinline__ int4 row_bytes(const int8_t* p, int64_t ld, int r, int rows, int k,
                                          int K) {
  if (r >= rows || k >= K) return make_int4(0, 0, 0, 0);
  const int8_t* s = p + static_cast<int64_t>(r) * ld + k;
  if (k + 16 <= K) return *reinterpret_cast<const int4*>(s);
  uint32_t w[4] = {0, 0, 0, 0};
  for (int i = 0; i < K - k; ++i)
    w[i / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(s[i])) << (8 * (i % 4));
  return make_int4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) linear_tile_kernel(const LinArgs a) {
  __shared__ int xs[kTile][kStepK / 4 + 1], ws[kTile][kStepK / 4 + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  int acc[4][4] = {};
  const int r = threadIdx.x / 4, kq = threadIdx.x % 4;
  for (int k0 = 0; k0 < a.K; k0 += kStepK) {
    const int4 xv = row_bytes(a.x, a.ldx, m0 + r, a.M, k0 + kq * 16, a.K);
    const int4 wv = row_bytes(a.w, a.ldw, n0 + r, a.N, k0 + kq * 16, a.K);
    __syncthreads();
    xs[r][kq * 4] = xv.x, xs[r][kq * 4 + 1] = xv.y, xs[r][kq * 4 + 2] = xv.z,
    xs[r][kq * 4 + 3] = xv.w;
    ws[r][kq * 4] = wv.x, ws[r][kq * 4 + 1] = wv.y, ws[r][kq * 4 + 2] = wv.z,
    ws[r][kq * 4 + 3] = wv.w;
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < kStepK / 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __dp4a(xs[ty + 16 * i][k], ws[tx + 16 * j][k], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      const float v = finish(a, acc[i][j], a.x_scale[m], a.w_scale[n],
                             a.bias != nullptr ? a.bias[n] : 0.f);
      if (a.y_bf16)
        static_cast<__nv_bfloat16*>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(v);
      else
        static_cast<float*>(a.y)[m * a.ldy + n] = v;
    }
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
  if (M < 0 || M > INT_MAX || N < 1 || N > INT_MAX || K < 1 || K > DLRM_INT8_MAX_K)
    return DLRM_ERR_SHAPE;
  if (ldx < K || ldw < K || ldy < N) return DLRM_ERR_SHAPE;
  if (w == nullptr || w_scale == nullptr) return DLRM_ERR_NULL;
  if (M > 0 && (x == nullptr || x_scale == nullptr || y == nullptr)) return DLRM_ERR_NULL;
  if (ldx % 16 != 0 || ldw % 16 != 0 || !is_aligned(x, 16) || !is_aligned(w, 16) ||
      !is_aligned(x_scale, 4) || !is_aligned(w_scale, 4) || !is_aligned(bias, 4) ||
      !is_aligned(y, dtype_size(y_dtype)) || !is_aligned(status_dev, 4))
    return DLRM_ERR_ALIGN;
  if (M == 0) return DLRM_OK;
  LinArgs a = {};
  a.x = x;
  a.w = w;
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.y = y;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldy = ldy;
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.act = act;
  a.y_bf16 = y_dtype == DLRM_TABLE_BF16;
  a.status = status_dev;
  const int64_t mt = (M + kTile - 1) / kTile;
  if (mt > 65535) return DLRM_ERR_SHAPE;
  linear_tile_kernel<<<dim3(static_cast<unsigned>((N + kTile - 1) / kTile),
                            static_cast<unsigned>(mt)),
                       256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  note_launch();
  return DLRM_OK;
}

}  // extern "C"
