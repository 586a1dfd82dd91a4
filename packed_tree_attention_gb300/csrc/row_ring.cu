// Launches of the kernels that stream rows of logits (row_ring.cuh).

#include "row_ring.cuh"

#include <algorithm>
#include <atomic>
#include <map>
#include <mutex>
#include <tuple>

namespace octo {
namespace rows {

// An attribute of the current device, asked for once.
template <cudaDeviceAttr kAttr>
static int attribute() {
  static std::atomic<int> known[64];   // + 1; devices past that are asked every time
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64)
    if (const int v = known[dev].load(std::memory_order_relaxed)) return v - 1;
  int n = 0;
  if (cudaDeviceGetAttribute(&n, kAttr, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

int sm_count() { return attribute<cudaDevAttrMultiProcessorCount>(); }
int64_t l2_bytes() { return attribute<cudaDevAttrL2CacheSize>(); }

int max_clusters(const void* kernel, int cs, int smem, int* out) {
  int dev = 0;
  OCTO_CUDA(cudaGetDevice(&dev));
  static std::mutex mu;
  static std::map<std::tuple<uintptr_t, int, int, int>, int> known;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(reinterpret_cast<uintptr_t>(kernel), dev, cs, smem);
  auto it = known.find(key);
  if (it != known.end()) {
    *out = it->second;
    return OCTO_OK;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs);
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  OCTO_CUDA(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg));
  known[key] = *out = std::max(1, n);
  return OCTO_OK;
}

int launch_overlapped(const void* kernel, const void* p, int grid, int block, int cs, int smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cs;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  void* args[1] = {const_cast<void*>(p)};
  OCTO_CUDA(cudaLaunchKernelExC(&cfg, kernel, args));
  count_launch();
  return OCTO_OK;
}

int launch_ring_raw(const void* kernel, const void* p, int32_t n, int cs, int smem, cudaStream_t s) {
  if (int st = set_smem_limit(kernel, kSmemMax)) return st;
  int clusters = sm_count();
  if (cs > 1)
    if (int st = max_clusters(kernel, cs, smem, &clusters)) return st;
  return launch_overlapped(kernel, p, (int)(std::min<int64_t>(n, std::max(1, clusters)) * cs), kBlock, cs, smem, s);
}

}  // namespace rows
}  // namespace octo
