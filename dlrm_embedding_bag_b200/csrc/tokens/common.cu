// Host-side bookkeeping of libdlrm_tokens.so.
#include <atomic>

#include "common.h"
#include "dlrm_tokens.h"

namespace dlrm {
namespace {

thread_local int t_last_cuda_error = 0;
std::atomic<int64_t> g_launches{0};

}  // namespace

int cuda_fail(cudaError_t e) {
  t_last_cuda_error = static_cast<int>(e);
  return DLRM_ERR_CUDA;
}

void note_launch(int n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

int sm_count_current() {
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cuda_fail(e);
    return 0;
  }
  return n;
}

EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

}  // namespace dlrm

extern "C" {

int dlrm_tokens_last_cuda_error(void) { return dlrm::t_last_cuda_error; }

int64_t dlrm_tokens_launch_count(void) {
  return dlrm::g_launches.load(std::memory_order_relaxed);
}

}  // extern "C"
