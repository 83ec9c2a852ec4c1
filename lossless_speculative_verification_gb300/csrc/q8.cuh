// q8.cuh -- sizes of the 8-bit form of rows and weights (q8.cu, q8mm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace lsv {

constexpr int kQ8Group = 128;      // columns (of a weight: rows and columns) that share a scale
constexpr int kQ8MaxCols = 16384;    // columns of a row
constexpr int kQ8MaxRows = 1 << 26;  // rows of a matrix

// Clusters of up to 8 CTAs of a kernel that a device holds at once (its SMs come in groups of uneven size); asked for once.
class ClustersAtOnce {
 public:
  // 0 on an error
  int of(const void* kernel, int size, int threads, int smem, int device) {
    int n = known_[device][size].load(std::memory_order_relaxed);
    if (n > 0) return n;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    known_[device][size].store(n, std::memory_order_relaxed);
    return n;
  }

 private:
  std::atomic<int> known_[64][9] = {};
};

// Loads of what an earlier kernel of the stream wrote.  A kernel that is launched before that one ends may not take
// them through the read-only path (what it loads must not change while it runs), which the compiler picks for
// const __restrict__ pointers: these are plain ones.
__device__ __forceinline__ uint4 ld_plain128(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// The same for what is read once.
__device__ __forceinline__ uint4 ld_stream128(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream64(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_plain_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

}  // namespace lsv
