// What the kernels on dense activations share (residual_norm.cu, adapter.cu,
// grad_clip.cu): element types, block sums, launches, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>
#include <utility>

#include "../../include/snack.h"

namespace snack {

void record_thread_error(const std::string &msg);  // api.cu
void count_launches(int n);                        // api.cu
int device_sms();                                  // SM count of the current device

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

// Rounds to nearest even: the one rounding of a stored result.
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// Two 16-bit elements in one register.
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t v, float &lo, float &hi);
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t v, float &lo, float &hi) {
  lo = __uint_as_float(v << 16);
  hi = __uint_as_float(v & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack2<__half>(uint32_t v, float &lo, float &hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
  lo = f.x;
  hi = f.y;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Element i of an array whose type is only known at run time.
__device__ __forceinline__ float load_as_float(const void *p, int type, int64_t i) {
  if (type == SNACK_F32) return static_cast<const float *>(p)[i];
  if (type == SNACK_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(static_cast<const __half *>(p)[i]);
}

__device__ __forceinline__ void store_from_float(void *p, int type, int64_t i, float v) {
  if (type == SNACK_F32)
    static_cast<float *>(p)[i] = v;
  else if (type == SNACK_BF16)
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// Programmatic dependent launches: a kernel launched with pdl waits for the
// whole of its predecessor here, before it touches any memory.
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependency_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over the block, the same in every thread; `red` holds
// N * 32 floats and may be reused after the call.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if (nw == 1) return;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 32 + w] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(lane < nw ? red[k * 32 + lane] : 0.f);
  __syncthreads();
}

// Asynchronous copies into shared memory (16-byte aligned global addresses);
// `bytes` below the size fills the rest with zeros.
__device__ __forceinline__ void copy_async16(void *slot, const void *from, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(slot)),
               "l"(from), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Lets the kernel be launched with that much dynamic shared memory, where it
// may be above the default (48 KB with the kernel's static part, at most 8 KB
// here).  The limit belongs to the kernel, not to the call: it is raised once,
// to all that a block can have, because a limit set to this call's size could
// be lowered by another host thread before the launch.
cudaError_t raise_smem_limit(const void *kern);  // dense_ops.cu
template <typename K>
inline cudaError_t allow_smem(K kern, size_t bytes) {
  return bytes <= 40 * 1024 ? cudaSuccess : raise_smem_limit(reinterpret_cast<const void *>(kern));
}

template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kern)(KArgs...), dim3 grid, int cluster, int threads, size_t smem, bool pdl,
                                   cudaStream_t s, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, bool pdl,
                                 cudaStream_t s, Args &&...args) {
  return launch_clusters(kern, grid, 1, threads, smem, pdl, s, std::forward<Args>(args)...);
}

inline snack_status refuse(snack_status st, const std::string &msg) {
  record_thread_error(msg);
  return st;
}

inline snack_status cuda_status(cudaError_t e, const char *what) {
  cudaGetLastError();  // reported here: not left for the caller's next CUDA call
  return refuse(e == cudaErrorMemoryAllocation ? SNACK_ERR_ALLOC : SNACK_ERR_CUDA,
                std::string(what) + ": " + cudaGetErrorString(e));
}

inline int64_t type_bytes(int type) { return type == SNACK_F32 ? 4 : 2; }
inline bool known_type(int type) { return type == SNACK_F32 || type == SNACK_BF16 || type == SNACK_F16; }
inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace snack
