// serving.cuh — device helpers of the serving-side operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "serving.h"

namespace dspark {

// Launches `kernel` so that it may start while its predecessor drains (it waits in
// griddep_wait() before its first access), as one-dimensional clusters of `cluster` CTAs.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster,
                           A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// SMs of the current device, asked once per device.
inline int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaGetDevice(&dev);
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n < 1) n = 1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Lets `kernel` use up to `bytes` of dynamic shared memory, set once per device and kernel:
// `done` (of the caller, one per kernel) remembers the devices.
template <typename F>
cudaError_t allow_smem(F* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  if (bytes <= 32 * 1024) return cudaSuccess;  // with the static part within the default 48 KB
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

__device__ __forceinline__ int ceil_div_dev(int a, int b) { return a / b + (a % b != 0); }

// 16-byte accesses of data that is read or written once.
__device__ __forceinline__ uint4 load_once16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void store16(void* p, uint4 v) {
  asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Inclusive sum over a block of up to 1024 threads of values in 0..kScanCap, held at kScanCap
// (which keeps the sum of two within 32 bits); `warp_sums` holds 32 ints.
constexpr int kScanCap = 1 << 24;
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, v, d);
    if (lane >= d) v = min(v + o, kScanCap);
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(~0u, w, d);
      if (lane >= d) w = min(w + o, kScanCap);
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  return min(v + (warp > 0 ? warp_sums[warp - 1] : 0), kScanCap);
}

// The first i in [0,n) with a[i] > x (n if none); a is non-decreasing.
__device__ __forceinline__ int upper_bound(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

}  // namespace dspark
