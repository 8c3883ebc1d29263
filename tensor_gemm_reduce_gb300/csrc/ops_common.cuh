// ops_common.cuh -- shared by the operators around the row-parallel layer:
// device check, launches and their status.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/gemm_rs_ops.h"
#include "ptx.cuh"

namespace grs {

// SMs of the current device if it is one this library is built for; looked up
// once for each device (a call costs tens of microseconds, a small operator
// takes a few).
inline int current_device_sms(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return GEMM_RS_ERR_UNSUPPORTED_DEVICE;
  }
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_RS_ERR_UNSUPPORTED_DEVICE;
    }
    if (major != 10 || minor != 3) return GEMM_RS_ERR_UNSUPPORTED_DEVICE;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return GEMM_RS_OK;
}

inline int launch_status() {
  return cudaGetLastError() == cudaSuccess ? GEMM_RS_OK : GEMM_RS_ERR_CUDA;
}

// More than 48 KB of dynamic shared memory for a kernel, asked for once on each
// device.
class SmemAllowed {
 public:
  template <typename Kernel>
  bool set(Kernel kernel, int bytes) {
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (done_.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    done_.fetch_or(bit, std::memory_order_relaxed);
    return true;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// Launch with programmatic dependent launch: the kernel's blocks may be placed
// while the previous kernel on the stream finishes.  Every kernel launched this
// way calls griddep_wait() before it touches global memory.
template <typename... P, typename... A>
int launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                      const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_RS_ERR_CUDA;
  }
  return GEMM_RS_OK;
}

inline bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Loads of what an earlier kernel may have written.  volatile, so that they stay
// behind griddep_wait(); the _stream forms are for data that is read once.
__device__ __forceinline__ uint4 load_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ float load_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_v4_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_v2_stream(const void* p) {
  uint2 v;
  asm volatile("ld.global.cs.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_u32_stream(const void* p) {
  uint32_t v;
  asm volatile("ld.global.cs.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_u16_stream(const void* p) {
  uint16_t v;
  asm volatile("ld.global.cs.b16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}

}  // namespace grs
