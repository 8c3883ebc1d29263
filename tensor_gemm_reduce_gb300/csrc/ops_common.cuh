// ops_common.cuh -- shared by the operators around the row-parallel layer:
// device check, launch status, bf16 vectors and block-wide sums.
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

inline bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16lo_to_f32(v.x); f[1] = bf16hi_to_f32(v.x);
  f[2] = bf16lo_to_f32(v.y); f[3] = bf16hi_to_f32(v.y);
  f[4] = bf16lo_to_f32(v.z); f[5] = bf16hi_to_f32(v.z);
  f[6] = bf16lo_to_f32(v.w); f[7] = bf16hi_to_f32(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 v;
  v.x = pack_bf16x2(f[0], f[1]);
  v.y = pack_bf16x2(f[2], f[3]);
  v.z = pack_bf16x2(f[4], f[5]);
  v.w = pack_bf16x2(f[6], f[7]);
  return v;
}

// Sum of each of the N values over the block, in every thread (the same bits
// in each: the butterfly adds the same pairs on both sides).  `part` holds
// 32 * N floats; a block alternates between two of them, so that one barrier
// a sum is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? part[i * 32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

}  // namespace grs
