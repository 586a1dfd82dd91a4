// Launches of the kernels that stream rows of logits (row_ring.cuh).

#include "row_ring.cuh"

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

namespace octo {
namespace rows {

int sm_count() {
  static std::mutex mu;
  static std::map<int, int> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  auto it = known.find(dev);
  if (it != known.end()) return it->second;
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return known[dev] = n;
}

int pick_cluster(int32_t n, int64_t nv, int ring_bytes, int rows_held) {
  const int sms = std::max(1, sm_count());
  int best = 1;
  double best_t = 0;
  for (int cs = 1; cs <= kMaxCluster; cs *= 2) {
    const int slots = std::max(1, sms / cs);
    const double rounds = (n + slots - 1) / slots;
    const double part = (double)((nv + cs - 1) / cs) * 16e-3;   // KB
    // an SM's share of the memory rate is 45 KB/us; alone it reaches about 80
    const double rate = 45.0 * std::min(1.8, std::max(1.0, (double)sms / ((double)std::min(n, slots) * cs)));
    const double t = rounds * (part / rate + 0.25 + (cs > 1 ? 0.15 : 0.0));
    if (cs == 1 || t < 0.97 * best_t) best = cs, best_t = t;
  }
  return best;
}

// Clusters of this kernel, size and shared memory that the device holds at once.
static int max_clusters(const void* kernel, int cs, int smem, int* out) {
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

int launch_ring_raw(const void* kernel, const void* p, int32_t n, int cs, int smem, cudaStream_t s) {
  if (int st = set_smem_limit(kernel, kSmemMax)) return st;
  int clusters = 0;
  if (cs == 1) clusters = std::max(1, sm_count());
  else if (int st = max_clusters(kernel, cs, smem, &clusters)) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(n, clusters) * cs));
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  void* args[1] = {const_cast<void*>(p)};
  OCTO_CUDA(cudaLaunchKernelExC(&cfg, kernel, args));
  count_launch();
  return OCTO_OK;
}

}  // namespace rows
}  // namespace octo
