// act8.cu -- 8-bit checkpoints of the row-parallel layer's input
// (gemm_rs_act8_* in include/gemm_rs_ops.h).
//
// A code byte holds the sign (bit 7) and the magnitude (bits 0..6), so that
// 128 + magnitude is one OR away from a bf16 (0x4300 | m): the backward pass
// rebuilds two elements at a time with bf16x2 arithmetic, all of it exact.
// The four bytes of a word hold elements 0, 2, 1, 3: the low bytes of its
// 16-bit halves are elements 0 and 1, the high ones 2 and 3.
// Both kernels move 3.03 bytes an element and are bound by HBM.
#include "act8.cuh"
#include "ops_common.cuh"

using namespace grs;

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 16;  // elements: 32 bytes of bf16, one 16-byte store of codes

struct Act8Params {
  long long rows;      // rows of `cols` elements, `pitch` codes apart
  long long cols, pitch;
  uint4* a;            // [rows][cols] bf16
  uint4* codes;        // [rows][pitch]
  uint8_t* scales;     // [rows][pitch / 32]
};

// A pair of threads shares a group: 16 elements each.
__global__ void __launch_bounds__(kThreads) act8_save_kernel(const Act8Params p) {
  const long long per_row = p.pitch / kPerThread;
  const long long units = p.rows * per_row;
  const long long stride = (long long)gridDim.x * kThreads;
  const int lane = threadIdx.x & 31;
  // whole warps stay in the loop: the exchange below takes all 32 lanes
  for (long long u = (long long)blockIdx.x * kThreads + threadIdx.x; u - lane < units; u += stride) {
    const long long row = p.rows == 1 ? 0 : u / per_row;
    const long long col = (u - row * per_row) * kPerThread;
    const bool in = u < units;
    uint32_t v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // a row is a whole number of 8-element vectors
      const uint4 q = in && col + 8 * h < p.cols ? __ldcs(p.a + (row * p.cols + col) / 8 + h)
                                           : make_uint4(0, 0, 0, 0);
      v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, v[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // a row has an even number of units
    if (!in) continue;
    // 127 = (1 + 126/128) 2^6: the scale's biased exponent is the largest
    // magnitude's less 6, one more if its fraction is above 126/128
    const uint32_t E = top >> 7;
    const uint32_t scale_byte = E == 255u ? 255u : (uint32_t)max((int)E - 6 + ((top & 127u) == 127u), 1);
    // at the very top of the range 64 * 2^122 would be 2^128
    const uint32_t most = scale_byte >= 249u ? 63u : 127u;
    const float inv = __uint_as_float((254u - min(scale_byte, 253u)) << 23);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // elements 4i .. 4i + 3
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t pair = v[2 * i + j / 2];
        const float f = j & 1 ? bf16hi_to_f32(pair) : bf16lo_to_f32(pair);
        // |f| inv + 2^23 rounds to nearest even at the units place
        const uint32_t m = __float_as_uint(fmaf(fabsf(f), inv, 8388608.f)) & 0xFFu;
        c[j] = min(m, most) | ((__float_as_uint(f) >> 24) & 0x80u);
        if (scale_byte == 255u) c[j] = 0;
      }
      w[i] = c[0] | (c[2] << 8) | (c[1] << 16) | (c[3] << 24);
    }
    p.codes[(row * p.pitch + col) / kPerThread] = make_uint4(w[0], w[1], w[2], w[3]);
    if ((col & 16) == 0) p.scales[(row * p.pitch + col) / kAct8Group] = (uint8_t)scale_byte;
  }
}

__global__ void __launch_bounds__(kThreads) act8_restore_kernel(const Act8Params p) {
  const long long per_row = p.pitch / kPerThread;
  const long long units = p.rows * per_row;
  const long long stride = (long long)gridDim.x * kThreads;
  for (long long u = (long long)blockIdx.x * kThreads + threadIdx.x; u < units; u += stride) {
    const long long row = p.rows == 1 ? 0 : u / per_row;
    const long long col = (u - row * per_row) * kPerThread;
    if (col >= p.cols) continue;
    const uint4 q = __ldcs(p.codes + (row * p.pitch + col) / kPerThread);
    const uint32_t s2 = act8_scale2(p.scales[(row * p.pitch + col) / kAct8Group]);
    const uint2 e0 = act8_restore4(q.x, s2), e1 = act8_restore4(q.y, s2), e2 = act8_restore4(q.z, s2),
                e3 = act8_restore4(q.w, s2);
    uint4* out = p.a + (row * p.cols + col) / 8;
    __stcs(out, make_uint4(e0.x, e0.y, e1.x, e1.y));
    if (col + 8 < p.cols) __stcs(out + 1, make_uint4(e2.x, e2.y, e3.x, e3.y));
  }
}

int check_shape(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || M % 8 || K % 64 || M > (1ll << 30) || K > (1ll << 30))
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

int run(bool save, int64_t M, int64_t K, void* A, void* codes, void* scales, void* stream) {
  int rc = check_shape(M, K);
  if (rc) return rc;
  if (M == 0 || K == 0) return GEMM_RS_OK;
  if (!A || !codes || !scales) return GEMM_RS_ERR_INVALID_ARG;
  if (misaligned16(A) || misaligned16(codes) || misaligned16(scales)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  Act8Params p;
  p.rows = kWorld8 * M;
  p.cols = K / kWorld8;
  p.pitch = act8_pitch(K / kWorld8);
  if (p.pitch == p.cols) {  // rows follow one another: one long row, no division by its length
    p.cols *= p.rows;
    p.pitch = p.cols;
    p.rows = 1;
  }
  p.a = static_cast<uint4*>(A);
  p.codes = static_cast<uint4*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  const long long blocks = (p.rows * p.pitch / kPerThread + kThreads - 1) / kThreads;
  const int grid = (int)(blocks < 16ll * sms ? blocks : 16ll * sms);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (save)
    act8_save_kernel<<<grid, kThreads, 0, st>>>(p);
  else
    act8_restore_kernel<<<grid, kThreads, 0, st>>>(p);
  return launch_status();
}

}  // namespace

extern "C" int gemm_rs_act8_layout(int64_t M, int64_t K, int64_t* pitch, size_t* code_bytes,
                                   size_t* scale_bytes) {
  const int rc = check_shape(M, K);
  if (rc) return rc;
  const int64_t pt = act8_pitch(K / kWorld8);
  if (pitch) *pitch = pt;
  if (code_bytes) *code_bytes = (size_t)kWorld8 * M * pt;
  if (scale_bytes) *scale_bytes = (size_t)kWorld8 * M * (pt / kAct8Group);
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_act8_save(int64_t M, int64_t K, const void* A, void* codes, void* scales,
                                 void* stream) {
  return run(true, M, K, const_cast<void*>(A), codes, scales, stream);
}

extern "C" int gemm_rs_act8_restore(int64_t M, int64_t K, const void* codes, const void* scales,
                                    void* A, void* stream) {
  return run(false, M, K, A, const_cast<void*>(codes), const_cast<void*>(scales), stream);
}
