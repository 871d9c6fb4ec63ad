// Launch of the persistent kernels that work in CTA pairs.
#pragma once
#include <atomic>

#include "internal.h"

namespace moe {

// `units` pieces of work on at most as many pairs as can be resident at once
// (one CTA per SM at either shared-memory size; the number is looked up once
// per kernel, and so is the shared-memory opt-in, per device).
template <typename Args>
cudaError_t launch_pairs(void (*kernel)(const Args), const Args& a, size_t smem, size_t smem_most,
                         int threads, long long units, const char* what, cudaStream_t st) {
  struct Known {
    std::atomic<const void*> kernel{nullptr};
    std::atomic<int> pairs{0};
    std::atomic<uint64_t> opted{0};  // devices
  };
  static Known known[8];
  Known* k = nullptr;
  for (Known& c : known) {
    const void* none = nullptr;
    if (c.kernel.load() == (const void*)kernel ||
        c.kernel.compare_exchange_strong(none, (const void*)kernel) ||
        none == (const void*)kernel) {
      k = &c;
      break;
    }
  }
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (k == nullptr || !(k->opted.load() & bit)) {
    const cudaError_t e =
        note_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem_most),
                  what);
    if (e != cudaSuccess) return e;
    if (k != nullptr) k->opted.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(num_sms() & ~1), 1, 1);
  int pairs = k != nullptr ? k->pairs.load() : 0;
  if (pairs == 0) {
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs <= 0)
      pairs = num_sms() / 2;
    if (k != nullptr) k->pairs.store(pairs);
  }
  if (units < pairs) pairs = (int)units;
  cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  return note_cuda(cudaLaunchKernelEx(&cfg, kernel, a), what);
}

}  // namespace moe
