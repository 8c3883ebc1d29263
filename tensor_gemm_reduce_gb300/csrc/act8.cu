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
constexpr int kUnroll = 2;      // units of 16 elements in flight for a thread

struct Act8Params {
  long long rows;      // rows of `cols` elements, `pitch` codes apart
  long long cols, pitch;
  uint4* a;            // [rows][cols] bf16
  uint4* codes;        // [rows][pitch]
  uint8_t* scales;     // [rows][pitch / 32]
};

// 16 elements of bf16.  kWide: 32-byte accesses (rows that follow one another and
// a 32-byte aligned tensor), so that a warp's access is 1 KiB in a row.
struct Sixteen {
  uint32_t v[8];
};
template <bool kWide>
__device__ __forceinline__ Sixteen load16(const uint4* p, bool first, bool second) {
  Sixteen r;
  if (kWide) {
    if (first)
      asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3]), "=r"(r.v[4]), "=r"(r.v[5]),
                     "=r"(r.v[6]), "=r"(r.v[7])
                   : "l"(p));
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) r.v[i] = 0;
    return r;
  }
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 a = first ? __ldcs(p) : none, b = second ? __ldcs(p + 1) : none;
  r.v[0] = a.x; r.v[1] = a.y; r.v[2] = a.z; r.v[3] = a.w;
  r.v[4] = b.x; r.v[5] = b.y; r.v[6] = b.z; r.v[7] = b.w;
  return r;
}
template <bool kWide>
__device__ __forceinline__ void store16(uint4* p, const Sixteen& r, bool second) {
  if (kWide) {
    asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.v[0]),
                 "r"(r.v[1]), "r"(r.v[2]), "r"(r.v[3]), "r"(r.v[4]), "r"(r.v[5]), "r"(r.v[6]), "r"(r.v[7])
                 : "memory");
    return;
  }
  __stcs(p, make_uint4(r.v[0], r.v[1], r.v[2], r.v[3]));
  if (second) __stcs(p + 1, make_uint4(r.v[4], r.v[5], r.v[6], r.v[7]));
}

// Where unit u (16 elements of a row) lies.
struct Place {
  long long a, code;  // element of A, byte of the codes
  bool first, second; // its two halves of 8 elements exist
};
__device__ __forceinline__ Place place_of(const Act8Params& p, long long u, long long units, long long per_row) {
  const long long row = p.rows == 1 ? 0 : u / per_row;
  const long long col = (u - row * per_row) * kPerThread;
  Place q;
  q.a = row * p.cols + col;
  q.code = row * p.pitch + col;
  q.first = u < units && col < p.cols;
  q.second = u < units && col + 8 < p.cols;
  return q;
}

// A pair of threads shares a group.  |a| / 2^e rounds to an integer m in the
// addition to 128 of one bf16x2 FMA, whose result is the pattern 0x4300 | m (in
// [128, 256) bf16 steps are 1, ties to even): the code without another step.
template <bool kWide>
__global__ void __launch_bounds__(kThreads) act8_save_kernel(const Act8Params p) {
  const long long per_row = p.pitch / kPerThread, units = p.rows * per_row;
  const long long stride = (long long)gridDim.x * kThreads;
  const int lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  // whole warps stay in the loop: the exchange below takes all 32 lanes
  for (long long u0 = (long long)blockIdx.x * kThreads + threadIdx.x; u0 - lane < units; u0 += kUnroll * stride) {
    Place at[kUnroll];
    Sixteen x[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      at[k] = place_of(p, u0 + k * stride, units, per_row);
      x[k] = load16<kWide>(p.a + at[k].a / 8, at[k].first, at[k].second);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      uint32_t mag[8], top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mag[i] = x[k].v[i] & 0x7FFF7FFFu;
        top = __vmaxu2(top, mag[i]);
      }
      top = max(top & 0xFFFFu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // a row has an even number of units
      if (u0 + k * stride >= units) continue;
      // 127 = (1 + 126/128) 2^6: the scale's biased exponent is the largest
      // magnitude's less 6, one more if its fraction is above 126/128
      const uint32_t E = top >> 7;
      const uint32_t scale = E == 255u ? 255u : (uint32_t)max((int)E - 6 + ((top & 127u) == 127u), 1);
      const uint32_t inv2 = ((254u - min(scale, 253u)) << 7) * 0x10001u;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // elements 4 i .. 4 i + 3
        const uint32_t lo = act8_round2(mag[2 * i], inv2), hi = act8_round2(mag[2 * i + 1], inv2);
        const uint32_t sign = ((x[k].v[2 * i] >> 8) & 0x00800080u) | (x[k].v[2 * i + 1] & 0x80008000u);
        w[i] = (lo & 0x007F007Fu) | ((hi << 8) & 0x7F007F00u) | sign;
      }
      if (scale >= 249u) {  // not finite, or so large that 64 * 2^122 would be 2^128
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = scale == 255u ? 0u : __vminu4(w[i] & 0x7F7F7F7Fu, 0x3F3F3F3Fu) | (w[i] & 0x80808080u);
      }
      p.codes[at[k].code / kPerThread] = make_uint4(w[0], w[1], w[2], w[3]);
      if ((lane & 1) == 0) p.scales[at[k].code / kAct8Group] = (uint8_t)scale;
    }
  }
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads) act8_restore_kernel(const Act8Params p) {
  const long long per_row = p.pitch / kPerThread, units = p.rows * per_row;
  const long long stride = (long long)gridDim.x * kThreads;
  griddep_launch_dependents();
  griddep_wait();
  for (long long u0 = (long long)blockIdx.x * kThreads + threadIdx.x; u0 < units; u0 += kUnroll * stride) {
    Place at[kUnroll];
    uint4 q[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      at[k] = place_of(p, u0 + k * stride, units, per_row);
      if (at[k].first) {
        q[k] = __ldcs(p.codes + at[k].code / kPerThread);
        s[k] = p.scales[at[k].code / kAct8Group];
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (!at[k].first) continue;
      const uint32_t s2 = act8_scale2(s[k]);
      const uint2 e0 = act8_restore4(q[k].x, s2), e1 = act8_restore4(q[k].y, s2), e2 = act8_restore4(q[k].z, s2),
                  e3 = act8_restore4(q[k].w, s2);
      store16<kWide>(p.a + at[k].a / 8, Sixteen{{e0.x, e0.y, e1.x, e1.y, e2.x, e2.y, e3.x, e3.y}}, at[k].second);
    }
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
  const bool wide = p.rows == 1 && (reinterpret_cast<uintptr_t>(A) & 31u) == 0;
  const long long blocks = (p.rows * p.pitch / kPerThread + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const int grid = (int)(blocks < 8ll * sms ? blocks : 8ll * sms);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launch_overlapped(save ? (wide ? act8_save_kernel<true> : act8_save_kernel<false>)
                                : (wide ? act8_restore_kernel<true> : act8_restore_kernel<false>),
                           dim3((unsigned)grid), kThreads, 0, st, p);
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
