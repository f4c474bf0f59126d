#include "dense_ops.cuh"

#include <mutex>
#include <set>

namespace snack {

cudaError_t raise_smem_limit(const void *kern) {
  static std::mutex lock;
  static std::set<std::pair<const void *, int>> raised;  // kernel, device
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const std::lock_guard<std::mutex> guard(lock);
  if (raised.count({kern, dev})) return cudaSuccess;
  cudaFuncAttributes at;
  if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)at.sharedSizeBytes);
  if (e == cudaSuccess) raised.insert({kern, dev});
  return e;
}

}  // namespace snack
