// act8.cu -- 8-bit checkpoints of the row-parallel layer's input
// (gemm_rs_act8_* in include/gemm_rs_ops.h).
//
// A code byte holds the sign (bit 7) and the magnitude (bits 0..6), so that
// 128 + magnitude is one OR away from a bf16 (0x4300 | m): the backward pass
// rebuilds two elements at a time with bf16x2 arithmetic, all of it exact.
// The four bytes of a word hold elements 0, 2, 1, 3: the low bytes of its
// 16-bit halves are elements 0 and 1, the high ones 2 and 3.
// Both kernels move 3.03 bytes an element and are bound by HBM: the two together take
// 214 us for 8192 x 28672 (1.42 GB, 6.64 TB/s, a copy's rate is 6.79) and 15.3 us for
// 512 x 28672 (5.8 TB/s).  Plain 16-byte loads, four in flight a thread and enough
// threads on each SM, reach that without shared memory.
#include "act8.cuh"
#include "ops_common.cuh"

using namespace grs;

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 8;  // elements: 16 bytes of bf16, 8 bytes of codes
constexpr int kUnroll = 4;     // units of 8 elements in flight for a thread
constexpr int kBlocksPerSm = 64;

// n / d for n < 2^31 as a multiplication (Granlund and Montgomery's method: with
// 2^(l-1) < d <= 2^l and mul = ceil(2^(31+l) / d) the error n (mul d - 2^(31+l)) is
// below 2^(31+l)).
struct Divider {
  uint32_t mul, shift;
};
Divider divider_of(uint32_t d) {
  Divider v = {0, 31};
  while (v.shift < 62 && (1ull << (v.shift - 31)) < d) ++v.shift;
  v.mul = (uint32_t)(((1ull << v.shift) + d - 1) / d);
  return v;
}

struct Act8Params {
  long long rows;      // rows of `cols` elements, `pitch` codes apart
  long long cols, pitch;
  Divider per_row;     // by the units of a row
  uint4* a;            // [rows][cols] bf16
  uint2* codes;        // [rows][pitch]
  uint8_t* scales;     // [rows][pitch / 32]
};

// Where unit u (8 elements of a row) lies.
struct Place {
  long long a, code;  // element of A, byte of the codes
  bool in;            // within the row (a row is a whole number of units, a pitch may hold more)
};
__device__ __forceinline__ Place place_of(const Act8Params& p, long long u, long long units) {
  long long row = 0;
  if (p.rows > 1)
    row = u < (1ll << 31) ? (long long)(((uint64_t)u * p.per_row.mul) >> p.per_row.shift) : u / (p.pitch / kPerThread);
  const long long col = u * kPerThread - row * p.pitch;
  return Place{row * p.cols + col, u * kPerThread, u < units && col < p.cols};
}

// Four threads share a group.  |a| / 2^e rounds to an integer m in the addition to
// 128 of one bf16x2 FMA, whose result is the pattern 0x4300 | m (in [128, 256)
// bf16 steps are 1, ties to even): the code without another step.
__global__ void __launch_bounds__(kThreads) act8_save_kernel(const Act8Params p) {
  const long long units = p.rows * (p.pitch / kPerThread);
  const long long stride = (long long)gridDim.x * kThreads;
  const int lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  // whole warps stay in the loop: the exchanges below take all 32 lanes
  for (long long u0 = (long long)blockIdx.x * kThreads + threadIdx.x; u0 - lane < units; u0 += kUnroll * stride) {
    Place at[kUnroll];
    uint4 x[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      at[k] = place_of(p, u0 + k * stride, units);
      x[k] = at[k].in ? load_v4_stream(p.a + at[k].a / kPerThread) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      uint32_t mag[4], top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mag[i] = v[i] & 0x7FFF7FFFu;
        top = __vmaxu2(top, mag[i]);
      }
      top = max(top & 0xFFFFu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // a pitch is a whole number of groups
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (u0 + k * stride >= units) continue;
      // 127 = (1 + 126/128) 2^6: the scale's biased exponent is the largest
      // magnitude's less 6, one more if its fraction is above 126/128
      const uint32_t E = top >> 7;
      const uint32_t scale = E == 255u ? 255u : (uint32_t)max((int)E - 6 + ((top & 127u) == 127u), 1);
      const uint32_t inv2 = ((254u - min(scale, 253u)) << 7) * 0x10001u;
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // elements 4 i .. 4 i + 3
        const uint32_t lo = act8_round2(mag[2 * i], inv2), hi = act8_round2(mag[2 * i + 1], inv2);
        const uint32_t sign = ((v[2 * i] >> 8) & 0x00800080u) | (v[2 * i + 1] & 0x80008000u);
        w[i] = (lo & 0x007F007Fu) | ((hi << 8) & 0x7F007F00u) | sign;
      }
      if (scale >= 249u) {  // not finite, or so large that 64 * 2^122 would be 2^128
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w[i] = scale == 255u ? 0u : __vminu4(w[i] & 0x7F7F7F7Fu, 0x3F3F3F3Fu) | (w[i] & 0x80808080u);
      }
      p.codes[at[k].code / kPerThread] = make_uint2(w[0], w[1]);
      if ((lane & 3) == 0) p.scales[at[k].code / kAct8Group] = (uint8_t)scale;
    }
  }
}

__global__ void __launch_bounds__(kThreads) act8_restore_kernel(const Act8Params p) {
  const long long units = p.rows * (p.pitch / kPerThread);
  const long long stride = (long long)gridDim.x * kThreads;
  griddep_wait();
  // only now: the backward kernel counts on every earlier kernel being complete
  // when it starts, and waits for this one where it needs it
  griddep_launch_dependents();
  for (long long u0 = (long long)blockIdx.x * kThreads + threadIdx.x; u0 < units; u0 += kUnroll * stride) {
    Place at[kUnroll];
    uint2 q[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      at[k] = place_of(p, u0 + k * stride, units);
      if (at[k].in) {
        q[k] = load_v2_stream(p.codes + at[k].code / kPerThread);
        s[k] = p.scales[at[k].code / kAct8Group];
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (!at[k].in) continue;
      const uint32_t s2 = act8_scale2(s[k]);
      const uint2 e0 = act8_restore4(q[k].x, s2), e1 = act8_restore4(q[k].y, s2);
      __stcs(p.a + at[k].a / kPerThread, make_uint4(e0.x, e0.y, e1.x, e1.y));
    }
  }
}

int check_shape(int64_t M, int64_t K) {
  if (M < 0 || K < 0 || M % 8 || K % 64 || M > (1ll << 30) || K > (1ll << 30))
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

// blocks_per_sm bounds the grid; padded: A's rows are as far apart as the codes'.
int run(bool save, int64_t M, int64_t K, void* A, void* codes, void* scales, void* stream, int blocks_per_sm,
        bool padded = false) {
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
  if (padded) p.cols = p.pitch;
  if (p.pitch == p.cols) {  // rows follow one another: one long row, no division by its length
    p.cols *= p.rows;
    p.pitch = p.cols;
    p.rows = 1;
  }
  p.per_row = divider_of(p.rows > 1 ? (uint32_t)(p.pitch / kPerThread) : 1u);
  p.a = static_cast<uint4*>(A);
  p.codes = static_cast<uint2*>(codes);
  p.scales = static_cast<uint8_t*>(scales);
  const long long blocks = (p.rows * p.pitch / kPerThread + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const int grid = (int)(blocks < (long long)blocks_per_sm * sms ? blocks : (long long)blocks_per_sm * sms);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_overlapped(save ? act8_save_kernel : act8_restore_kernel, dim3((unsigned)grid), kThreads, 0, st, p);
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
  return run(true, M, K, const_cast<void*>(A), codes, scales, stream, kBlocksPerSm);
}

extern "C" int gemm_rs_act8_restore(int64_t M, int64_t K, const void* codes, const void* scales,
                                    void* A, void* stream) {
  return run(false, M, K, A, const_cast<void*>(codes), const_cast<void*>(scales), stream, kBlocksPerSm);
}

int grs::act8_restore_padded(int64_t M, int64_t K, const void* codes, const void* scales, void* A, bool beside,
                             void* stream) {
  return run(false, M, K, A, const_cast<void*>(codes), const_cast<void*>(scales), stream, beside ? 2 : kBlocksPerSm, true);
}
