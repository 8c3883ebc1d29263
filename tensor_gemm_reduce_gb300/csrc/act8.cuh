// act8.cuh -- the format of 8-bit checkpoints, shared by the kernels that
// write, restore and multiply them (see act8.cu).
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace grs {

constexpr int kWorld8 = 8;
constexpr int kAct8Group = 32;  // elements of a row that share a scale

// Codes of a row of `cols` elements, in whole 128-byte lines.
inline int64_t act8_pitch(int64_t cols) { return (cols + 127) / 128 * 128; }

// gemm_rs_act8_restore into rows act8_pitch(K / 8) elements apart, zero beyond
// the row's end.  `beside`: with two blocks an SM, which leave room for a block of
// the backward kernel; that kernel may start before this one has ended.
int act8_restore_padded(int64_t M, int64_t K, const void* codes, const void* scales, void* A, bool beside,
                        void* stream);

// Scale byte b stands for 2^(b - 127), whose bf16 pattern is b << 7; 255 gives
// infinity, and its group's codes are zero, so their product is NaN.  Byte 0
// (only read beyond the rows and columns there are) gives 0.
__device__ __forceinline__ uint32_t act8_scale2(uint32_t b) { return (b << 7) * 0x10001u; }

// Two magnitudes times `inv2` (a power of two, at most 127 as products), rounded
// to nearest even, as 0x4300 | m.
__device__ __forceinline__ uint32_t act8_round2(uint32_t mag, uint32_t inv2) {
  const uint32_t k128 = 0x43004300u;
  const __nv_bfloat162 r =
      __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&mag), *reinterpret_cast<const __nv_bfloat162*>(&inv2),
              *reinterpret_cast<const __nv_bfloat162*>(&k128));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four code bytes to four bf16, elements 0, 1 in .x and 2, 3 in .y:
// (128 + m) - 128 and the product with a power of two are exact in bf16.
__device__ __forceinline__ uint32_t act8_magnitude2(uint32_t m, uint32_t scale2) {
  const uint32_t k128 = 0x43004300u;
  const uint32_t t = m | k128;
  __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&t);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&k128);
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&scale2);
  a = __hmul2(__hsub2(a, b), s);
  return *reinterpret_cast<const uint32_t*>(&a);
}
__device__ __forceinline__ uint2 act8_restore4(uint32_t w, uint32_t scale2) {
  uint2 r;
  r.x = act8_magnitude2(w & 0x007F007Fu, scale2) | ((w << 8) & 0x80008000u);
  r.y = act8_magnitude2((w >> 8) & 0x007F007Fu, scale2) | (w & 0x80008000u);
  return r;
}

}  // namespace grs
