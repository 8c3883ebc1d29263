// fp8.cu -- the row-parallel layer in 8-bit floating point (gemm_rs_fp8_* in
// include/gemm_rs_ops.h): quantisation to e4m3 with a scale for each block of 128,
// and the layer's forward and backward pass from such codes.
//
// A block's scale is its largest magnitude over 448, e4m3's largest, in fp32; a code is the
// element times the scale's reciprocal, rounded to nearest even.  Where the caller asks for it, it is
// the least power of two, from 2^-126 on, whose 448-fold is no less than the largest magnitude, which
// the tensor cores apply by themselves: 2048 x 8192 x 8192 forward takes 93 us for 139.  It costs accuracy, as a
// block's largest then lies anywhere in the upper octave of the codes and off their grid: inputs with one
// entry in 20 eight times as large are rounded by 2.7% of their norm, with fp32 by 2.1%.  Blocks are
// 128 x 128 for weights, 128 elements along the inner dimension of the product for activations
// and gradients: along a row for the forward pass and dA, along 128 tokens for dW.
#include <cstring>

#include "fp8.cuh"

using namespace grs;

namespace {

constexpr int kThreads = 256;
constexpr int kPairs = 76;  // of a GB300's SMs
// fp32 of 1 / 448, and the least magnitude that a block's largest counts as: an fp32 scale and its
// reciprocal are normal numbers.
constexpr float kPerLargest = (float)(1.0 / 448.0);
constexpr float kSmallest = 7.888609052210118e-31f;  // 2^-100

struct QuantizeParams {
  const uint4* x;
  long long x_plane;  // vectors of 8 between planes of x
  int vec;            // vectors in a row
  int M, experts, cb, rb, planes, span;
  const int* offsets;
  const int* pairs;
  const float* weights;
  int top_k;
  uint2* row_codes;
  void* row_scales;
  long long row_pitch;  // of row_scales: words for a block, bytes' words for four
  uint2* token_codes;
  void* token_scales;
  long long padded;  // rows of token_codes in a plane
  int code_vec;                   // pitch of codes in vectors of 8
  uint32_t* status;
};

// The scale's biased exponent for a block whose largest magnitude has these fp32 bits:
// 448 = 1.75 * 2^8.  Infinities and NaN, as integers above every finite magnitude: 255.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u);
  return top >= 0x7F800000u ? 255u : (uint32_t)max(e, 1);
}
// 1 / scale, a power of two; NaN for 255.
__device__ __forceinline__ float inverse_of(uint32_t scale) {
  return __uint_as_float(scale == 255u ? 0x7FC00000u : (254u - scale) << 23);
}

// The fp32 scale; NaN for infinities and NaN.
__device__ __forceinline__ float scale_f32(uint32_t top) {
  const float scale = fmaxf(__uint_as_float(top), kSmallest) * kPerLargest;
  return top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : scale;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The expert whose block of 128 rows `rb` is, its first row in that block and the row
// behind its last; blocks are counted expert by expert.  All threads of the CTA.
__device__ __forceinline__ bool find_block(const int* offsets, int experts, int M, int rb, int* row0, int* end) {
  __shared__ int sums[kThreads / 32], found[2];
  const int tid = threadIdx.x, lane = tid & 31;
  int first = 0, last = 0;
  if (tid < experts) {
    first = expert_row(offsets, tid, M);
    last = expert_row(offsets, tid + 1, M);
  }
  const int n = last > first ? (last - first + kBlk - 1) / kBlk : 0;
  int sum = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 31) sums[tid >> 5] = sum;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  for (int w = 0; w < (tid >> 5); ++w) sum += sums[w];
  if (rb >= sum - n && rb < sum) {
    found[0] = first + (rb - (sum - n)) * kBlk;
    found[1] = last;
  }
  __syncthreads();
  *row0 = found[0];
  *end = found[1];
  return found[0] >= 0;
}

// Largest magnitudes of pairs of bf16, as integers.
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
__device__ __forceinline__ uint32_t top_pair(uint4 x) {
  return max_pairs(max_pairs(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), max_pairs(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
}

// scale_of for a bf16 pattern, and 1 / scale as bf16: a product by it is exact (what leaves
// bf16's normal range below rounds to zero in e4m3 in any case).
__device__ __forceinline__ uint32_t scale_of_bf16(uint32_t top) {
  const int e = (int)(top >> 7) - 8 + ((top & 0x7Fu) > 0x60u);
  return top >= 0x7F80u ? 255u : (uint32_t)max(e, 1);
}
__device__ __forceinline__ uint32_t inverse_bf16(uint32_t scale) { return scale == 255u ? 0x7FC0u : (254u - scale) << 7; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Codes of four elements, pairs by pairs times their inverse scales.
__device__ __forceinline__ uint32_t scaled4(uint32_t x, uint32_t ix, uint32_t y, uint32_t iy) {
  x = mul_bf16x2(x, ix);
  y = mul_bf16x2(y, iy);
  return codes4(bf16lo_to_f32(x), bf16hi_to_f32(x), bf16lo_to_f32(y), bf16hi_to_f32(y));
}

__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t product_codes4(uint64_t x, uint64_t ix, uint64_t y, uint64_t iy) {
  x = mul_f32x2(x, ix);
  y = mul_f32x2(y, iy);
  return codes4(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)), __uint_as_float((uint32_t)y),
                __uint_as_float((uint32_t)(y >> 32)));
}

// Codes of four bf16 elements, pairs by pairs times their inverse scales in fp32.
__device__ __forceinline__ uint32_t scaled4_f32(uint32_t x, uint64_t ix, uint32_t y, uint64_t iy) {
  return product_codes4(pack_f32x2(bf16lo_to_f32(x), bf16hi_to_f32(x)), ix, pack_f32x2(bf16lo_to_f32(y), bf16hi_to_f32(y)), iy);
}

// A CTA's tile is 128 rows x 128 columns: a thread holds 8 columns of 8 rows, 16 rows
// apart.  x is read once for both kinds of codes.  Bound by memory: 8192 x 28672 by rows
// 100 us (7.0 TB/s), 4096 x 16384 of 8 experts both ways 52 us (5.1 TB/s).  Rows that are gathered
// and weighted take `span` tiles a CTA, so that finding them is paid once (4096 x 6144: 42 us
// with one, 29 with four).
template <bool kRows, bool kTokens, bool kGather, bool kE8m0>
__global__ void __launch_bounds__(kThreads, kGather ? 2 : kTokens ? 3 : 4) quantize_kernel(const QuantizeParams p) {
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int spans = kGather ? (p.cb + p.span - 1) / p.span : p.cb;
  const int cb0 = blockIdx.x % spans * (kGather ? p.span : 1), rest = blockIdx.x / spans;
  const int rb = rest % p.rb, plane = rest / p.rb;
  griddep_wait();
  // only now: the product for few rows asks for weights as soon as it may start, and counts
  // on everything before this launch being complete
  griddep_launch_dependents();
  if (blockIdx.x == 0 && tid == 0 && p.status) *p.status = 0;
  int row0 = rb * kBlk, end = p.M;
  if (p.offsets) {
    if constexpr (kTokens) {
      if (!find_block(p.offsets, p.experts, p.M, rb, &row0, &end)) return;
    } else {
      end = expert_row(p.offsets, p.experts, p.M);
    }
  }
  if (row0 >= end) return;
  const int half0 = tid & 16;  // first lane of this half-warp, whose lanes share rows
  float weight[8];
  int source[8];
  if constexpr (kGather) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = row0 + ty + 16 * i, pair = p.pairs[row < end ? row : row0];
      const bool valid = row < end && (unsigned)pair < (unsigned)p.M;
      weight[i] = valid ? p.weights[pair] : 0.f;
      source[i] = valid ? pair / p.top_k : -1;
    }
  }
  const int cb1 = kGather && cb0 + p.span < p.cb ? cb0 + p.span : kGather ? p.cb : cb0 + 1;
  for (int cb = cb0; cb < cb1; ++cb) {
    const int col = cb * 16 + tx;  // vector of 8 columns
    const bool in = col < p.vec;
    uint4 raw[8];
    uint64_t prod[kGather ? 8 : 1][4];  // rows that are weighted: the products, pairs of fp32
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = row0 + ty + 16 * i;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (row < end && in) {
        if constexpr (kGather) {
          if (source[i] >= 0) raw[i] = load_v4(p.x + (long long)source[i] * p.vec + col);  // top_k rows read it
        } else {
          raw[i] = load_v4_stream(p.x + plane * p.x_plane + (long long)row * p.vec + col);
        }
      }
    }
    if constexpr (kGather) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          prod[i][j] = mul_f32x2(pack_f32x2(bf16lo_to_f32(w[j]), bf16hi_to_f32(w[j])), pack_f32x2(weight[i], weight[i]));
      }
    }
    if constexpr (kRows) {
      // 16 lanes share a row: two rows' largest in a word
      uint32_t top[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t t0 = top_pair(raw[2 * i]), t1 = top_pair(raw[2 * i + 1]);
        top[i] = max_pairs(__byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632));
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = max_pairs(top[i], __shfl_xor_sync(0xffffffffu, top[i], d));
      // lane i of 8 works out row i's scale, and hands its inverse to the others
      const int mine = tx & 7;
      uint32_t word = mine & 4 ? (mine & 2 ? top[3] : top[2]) : (mine & 2 ? top[1] : top[0]);
      word = mine & 1 ? word >> 16 : word & 0xFFFFu;
      word <<= 16;
      if constexpr (kGather) {
        float w = weight[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) w = mine == i ? weight[i] : w;
        // products by a weight are in the order of their factors
        word = __float_as_uint(__fmul_rn(__uint_as_float(word), w)) & 0x7FFFFFFFu;
      }
      uint32_t inverse;  // as fp32; for bytes and rows that are not weighted as a pair of bf16
      const int my_row = row0 + ty + 16 * mine, block = plane * p.cb + cb;
      const bool stores = tx < 8 && my_row < end;
      if constexpr (kE8m0) {
        const uint32_t scale = scale_of(word);
        inverse = kGather ? __float_as_uint(inverse_of(scale)) : inverse_bf16(scale) * 0x10001u;
        if (stores)
          static_cast<uint8_t*>(p.row_scales)[((block >> 2) * p.row_pitch + my_row) * 4 + (block & 3)] = (uint8_t)scale;
      } else {
        const float scale = scale_f32(word);
        inverse = __float_as_uint(__frcp_rn(scale));
        if (stores) static_cast<float*>(p.row_scales)[block * p.row_pitch + my_row] = scale;
      }
      uint2* out = p.row_codes + ((long long)plane * p.M + row0 + ty) * p.code_vec + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t inv = __shfl_sync(0xffffffffu, inverse, half0 + i);
        if (row0 + ty + 16 * i >= end || !in) continue;
        uint2 codes;
        const uint64_t f = pack_f32x2(__uint_as_float(inv), __uint_as_float(inv));
        if constexpr (kGather) {
          codes = make_uint2(product_codes4(prod[i][0], f, prod[i][1], f), product_codes4(prod[i][2], f, prod[i][3], f));
        } else if constexpr (!kE8m0) {
          codes = make_uint2(scaled4_f32(raw[i].x, f, raw[i].y, f), scaled4_f32(raw[i].z, f, raw[i].w, f));
        } else {
          codes = make_uint2(scaled4(raw[i].x, inv, raw[i].y, inv), scaled4(raw[i].z, inv, raw[i].w, inv));
        }
        out[(long long)(16 * i) * p.code_vec] = codes;
      }
    }
    if constexpr (kTokens) {
      // each warp's largest of its 16 rows, then a column's by one thread
      const int warp = tid >> 5;
      uint2* out = p.token_codes + ((long long)plane * p.padded + rb * kBlk + ty) * p.code_vec + col;
      // the first column's: a byte for every fourth, or fp32 each
      uint8_t* bytes = static_cast<uint8_t*>(p.token_scales) + ((long long)(rb >> 2) * p.planes + plane) * p.code_vec * 32 + (rb & 3);
      float* floats = static_cast<float*>(p.token_scales) + ((long long)rb * p.planes + plane) * p.code_vec * 8;
      if constexpr (kGather) {
        __shared__ uint32_t tops[kThreads / 32][kBlk];
        __shared__ float inverse[kBlk];
        uint32_t top[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            top[j] = max(top[j], (uint32_t)(prod[i][j >> 1] >> (32 * (j & 1))) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
          if (half0 == 0) tops[warp][j * 16 + tx] = top[j];
        }
        __syncthreads();
        if (tid < kBlk) {  // column 8 (tid % 16) + tid / 16 of the tile
          uint32_t t = 0;
#pragma unroll
          for (int w = 0; w < kThreads / 32; ++w) t = max(t, tops[w][tid]);
          if constexpr (kE8m0) {
            const uint32_t scale = scale_of(t);
            inverse[tid] = inverse_of(scale);
            if (in) bytes[(col * 8 + ty) * 4ll] = (uint8_t)scale;
          } else {
            const float scale = scale_f32(t);
            inverse[tid] = __frcp_rn(scale);
            if (in) floats[col * 8 + ty] = scale;
          }
        }
        __syncthreads();
        if (in) {
          uint64_t inv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) inv[j] = pack_f32x2(inverse[2 * j * 16 + tx], inverse[(2 * j + 1) * 16 + tx]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            out[(long long)(16 * i) * p.code_vec] = make_uint2(product_codes4(prod[i][0], inv[0], prod[i][1], inv[1]),
                                                               product_codes4(prod[i][2], inv[2], prod[i][3], inv[3]));
        }
      } else {
        __shared__ __align__(16) uint32_t tops[kThreads / 32][kBlk / 2];  // pairs of columns
        __shared__ __align__(16) uint32_t inverse[kE8m0 ? kBlk / 2 : kBlk];  // pairs of bf16, or fp32
        uint32_t top[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = max_pairs(top[j], w[j] & 0x7FFF7FFFu);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) top[j] = max_pairs(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
        if (half0 == 0) *reinterpret_cast<uint4*>(&tops[warp][4 * tx]) = make_uint4(top[0], top[1], top[2], top[3]);
        __syncthreads();
        if (tid < kBlk / 2) {
          uint32_t t = 0;
#pragma unroll
          for (int w = 0; w < kThreads / 32; ++w) t = max_pairs(t, tops[w][tid]);
          const int c = cb * kBlk + 2 * tid;
          if constexpr (kE8m0) {
            const uint32_t lo = scale_of_bf16(t & 0xFFFFu), hi = scale_of_bf16(t >> 16);
            inverse[tid] = inverse_bf16(lo) | inverse_bf16(hi) << 16;
            if (c < p.vec * 8) {
              bytes[c * 4ll] = (uint8_t)lo;
              bytes[c * 4ll + 4] = (uint8_t)hi;
            }
          } else {
            const float lo = scale_f32(t << 16), hi = scale_f32(t & 0xFFFF0000u);
            inverse[2 * tid] = __float_as_uint(__frcp_rn(lo));
            inverse[2 * tid + 1] = __float_as_uint(__frcp_rn(hi));
            if (c < p.vec * 8) *reinterpret_cast<float2*>(floats + c) = make_float2(lo, hi);
          }
        }
        __syncthreads();
        if (in && !kE8m0) {
          uint64_t inv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            inv[j] = pack_f32x2(__uint_as_float(inverse[8 * tx + 2 * j]), __uint_as_float(inverse[8 * tx + 2 * j + 1]));
#pragma unroll
          for (int i = 0; i < 8; ++i)
            out[(long long)(16 * i) * p.code_vec] = make_uint2(scaled4_f32(raw[i].x, inv[0], raw[i].y, inv[1]),
                                                               scaled4_f32(raw[i].z, inv[2], raw[i].w, inv[3]));
        }
        if (in && kE8m0) {
          const uint4 inv = *reinterpret_cast<const uint4*>(&inverse[4 * tx]);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            out[(long long)(16 * i) * p.code_vec] = make_uint2(scaled4(raw[i].x, inv.x, raw[i].y, inv.y),
                                                               scaled4(raw[i].z, inv.z, raw[i].w, inv.w));
        }
      }
    }
    if constexpr (kGather && kTokens) __syncthreads();  // the shared maxima and inverses are used again
  }
}

template <bool kE8m0>
auto quantizer(bool gather, bool rows, bool tokens) {
  return gather ? (tokens ? (rows ? quantize_kernel<true, true, true, kE8m0> : quantize_kernel<false, true, true, kE8m0>)
                          : quantize_kernel<true, false, true, kE8m0>)
                : (tokens ? (rows ? quantize_kernel<true, true, false, kE8m0> : quantize_kernel<false, true, false, kE8m0>)
                          : quantize_kernel<true, false, false, kE8m0>);
}

// Weights: one scale for the CTA's 128 x 128 tile, whose codes are 16 KB in a row (rows of 128
// bytes, 8 KB apart in a weight of 8192 columns, were read at 4.7 TB/s where SMs read
// different parts of it).  Bound by memory: 8 x 16384 x 6144 332 us, 7.3 TB/s.
struct WeightParams {
  const uint4* w;
  uint2* codes;
  void* scales;
  int Kr, vec, kb, nb;
};

template <bool kE8m0>
__global__ void __launch_bounds__(kThreads) quantize_weight_kernel(const WeightParams p) {
  __shared__ uint32_t tops[kThreads / 32];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const long long block = blockIdx.x;
  const int nb = (int)(block % p.nb);
  const long long rest = block / p.nb;
  const int kb = (int)(rest % p.kb);
  const long long plane = rest / p.kb;
  griddep_launch_dependents();
  griddep_wait();
  const int col = nb * 16 + tx, row0 = kb * kBlk;
  const bool in = col < p.vec;
  uint4 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = row0 + ty + 16 * i;
    raw[i] = in && row < p.Kr ? load_v4_stream(p.w + (plane * p.Kr + row) * p.vec + col) : make_uint4(0, 0, 0, 0);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
  }
  top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, tops[w]);
  uint32_t inv;  // a pair of bf16, or fp32
  if constexpr (kE8m0) {
    const uint32_t scale = scale_of_bf16(top);
    inv = inverse_bf16(scale) * 0x10001u;
    if (tid == 0) static_cast<uint8_t*>(p.scales)[block] = (uint8_t)scale;
  } else {
    const float scale = scale_f32(top << 16);
    inv = __float_as_uint(__frcp_rn(scale));
    if (tid == 0) static_cast<float*>(p.scales)[block] = scale;
  }
  const uint64_t f = pack_f32x2(__uint_as_float(inv), __uint_as_float(inv));
  // the block's rows follow one another; columns behind the last are zero
  uint2* out = p.codes + ((plane * p.nb + nb) * p.Kr + row0) * 16 + tid;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (row0 + ty + 16 * i < p.Kr)
      out[256 * i] = kE8m0 ? make_uint2(scaled4(raw[i].x, inv, raw[i].y, inv), scaled4(raw[i].z, inv, raw[i].w, inv))
                           : make_uint2(scaled4_f32(raw[i].x, f, raw[i].y, f), scaled4_f32(raw[i].z, f, raw[i].w, f));
}

// Parts that the contraction of a forward pass is cut in where its tiles are few: of those that run
// at once (kPairs is a GB300's, as the size of a workspace does not ask the device) the number that saves most,
// 0.29 us a block of 128 (0.45 with fp32 scales, which would cut a few more) against 4 us for the launch that
// adds the parts up and the time to write and read them in fp32.  256 x 256 x 28672 68 -> 22 us, 277 x 176 x 5440 20 -> 17.
int parts_of(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256), steps = kWorld * blocks_of(K / kWorld);
  int best = 1;
  int64_t most = 0;
  for (int parts = 2; parts <= 8 && parts * tiles <= kPairs && parts <= steps; ++parts) {
    const int64_t saved = steps * (parts - 1) / parts * 29 - 400 - parts * M * N * 8 / 50000;  // units of 10 ns
    if (saved > most) {
      most = saved;
      best = parts;
    }
  }
  return best;
}

// out = the sum of the parts, in their order.
struct SumParams {
  const float* parts;
  uint4* out;
  long long vec;  // of 8 elements in a part
  int count;
};

__global__ void __launch_bounds__(kThreads) sum_parts_kernel(const SumParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.vec) return;
  float sum[8] = {};
#pragma unroll 8
  for (int c = 0; c < p.count; ++c) {
    const float* src = p.parts + (c * p.vec + i) * 8;
    const uint4 a = load_v4_stream(src), b = load_v4_stream(src + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += __uint_as_float(w[j]);
  }
  p.out[i] = make_uint4(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]), pack_bf16x2(sum[4], sum[5]),
                        pack_bf16x2(sum[6], sum[7]));
}

int check_shape(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || N % 8 || K % 64) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return fp8_check_sizes(M, 1, N, K);
}

template <typename T>
T* at(void* base, size_t bytes) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + bytes);
}

// Places in the workspace of a dense call.
struct Places {
  size_t row_codes, row_scales, token_codes, token_scales, parts, total;
};
Places forward_places(int64_t M, int64_t N, int64_t K) {
  const int64_t Kr = K / kWorld;
  Places w = {};
  w.row_codes = kFp8Status;
  w.row_scales = w.row_codes + align256((size_t)kWorld * M * fp8_pitch(Kr));
  w.parts = w.row_scales + align256(row_scale_bytes(M, kWorld * blocks_of(Kr)));
  const int parts = parts_of(M, N, K);
  w.total = w.parts + (parts > 1 ? (size_t)parts * M * N * 4 : 0);
  return w;
}
Places backward_places(int64_t M, int64_t N) {
  Places w = {};
  w.row_codes = kFp8Status;
  w.row_scales = w.row_codes + align256((size_t)M * fp8_pitch(N));
  w.token_codes = w.row_scales + align256(row_scale_bytes(M, blocks_of(N)));
  w.token_scales = w.token_codes + align256((size_t)padded_rows(M, 1) * fp8_pitch(N));
  w.total = w.token_scales + align256(token_scale_bytes(padded_rows(M, 1), 1, N));
  return w;
}

int clear(void* p, size_t bytes, cudaStream_t st) {
  if (bytes == 0) return GEMM_RS_OK;
  if (!p) return GEMM_RS_ERR_INVALID_ARG;
  if (cudaMemsetAsync(p, 0, bytes, st) == cudaSuccess) return GEMM_RS_OK;
  cudaGetLastError();
  return GEMM_RS_ERR_CUDA;
}

}  // namespace

int grs::fp8_check_sizes(int64_t M, int64_t experts, int64_t N, int64_t K) {
  // TMA coordinates, tile and block indices are 32-bit
  const int64_t Kr = K / kWorld, most = 1ll << 30;
  if (M > most / 2 || N > most || Kr > most || experts < 1 || experts > kMaxExperts) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  const int64_t mb = blocks_of(M) + experts, nb = blocks_of(N) + 1, kb = kWorld * (blocks_of(Kr) + 1);
  if (kb * experts > most / nb || mb > most / nb || mb > most / kb) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

int grs::fp8_quantize_rows(const Fp8Quantize& q, cudaStream_t st) {
  QuantizeParams p;
  memset(&p, 0, sizeof(p));
  const bool gather = q.rows.pairs != nullptr, rows = q.row_codes != nullptr, tokens = q.token_codes != nullptr;
  p.x = static_cast<const uint4*>(q.x);
  p.vec = (int)(q.cols / 8);
  p.x_plane = q.rows.M * p.vec;  // one plane where rows are gathered
  p.M = (int)q.rows.M;
  p.experts = q.rows.experts;
  p.offsets = q.rows.offsets;
  p.pairs = q.rows.pairs;
  p.weights = q.rows.weights;
  p.top_k = q.rows.top_k;
  p.cb = (int)blocks_of(q.cols);
  p.planes = q.planes;
  p.padded = padded_rows(q.rows.M, q.rows.offsets ? q.rows.experts : 1);
  p.rb = (int)(tokens ? p.padded / kBlk : blocks_of(q.rows.M));
  p.row_codes = static_cast<uint2*>(q.row_codes);
  p.row_scales = q.row_scales;
  p.row_pitch = row_scale_pitch(q.rows.M);
  p.token_codes = static_cast<uint2*>(q.token_codes);
  p.token_scales = q.token_scales;
  p.code_vec = (int)(fp8_pitch(q.cols) / 8);
  p.status = q.status;
  p.span = 1;
  if (gather) {  // about two CTAs an SM, of up to 4 tiles each
    int sms = 0;
    const int rc = current_device_sms(&sms);
    if (rc) return rc;
    const int64_t span = (int64_t)p.rb * p.cb / (2 * sms);
    p.span = (int)(span < 1 ? 1 : span > 4 ? 4 : span);
  }
  const dim3 grid((unsigned)((int64_t)p.planes * p.rb * ((p.cb + p.span - 1) / p.span)));
  const bool e8m0 = q.scale == kFp8E8m0;
  auto kernel = e8m0 ? quantizer<true>(gather, rows, tokens) : quantizer<false>(gather, rows, tokens);
  return launch_overlapped(kernel, grid, kThreads, 0, st, p);
}

namespace {

int weight_bytes(Fp8Scale scale, int64_t experts, int64_t N, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  if (N < 0 || K < 0 || N % 8 || K % 64) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  const int rc = fp8_check_sizes(0, experts, N, K);
  if (rc) return rc;
  const int64_t Kr = K / kWorld;
  if (code_bytes) *code_bytes = (size_t)experts * K * blocks_of(N) * kBlk;
  if (scale_bytes) *scale_bytes = (size_t)experts * kWorld * blocks_of(Kr) * blocks_of(N) * (scale == kFp8F32 ? 4 : 1);
  return GEMM_RS_OK;
}

// fp32 scales are aligned as every buffer is; bytes may lie anywhere.
bool misaligned_scales(Fp8Scale scale, const void* scales) { return scale == kFp8F32 && misaligned16(scales); }

int quantize(Fp8Scale scale, int64_t experts, int64_t N, int64_t K, const void* W, void* codes, void* scales, void* stream) {
  size_t bytes = 0;
  int rc = weight_bytes(scale, experts, N, K, &bytes, nullptr);
  if (rc) return rc;
  if (bytes == 0) return GEMM_RS_OK;
  if (!W || !codes || !scales) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {W, (const void*)codes})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (misaligned_scales(scale, scales)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  WeightParams p;
  p.w = static_cast<const uint4*>(W);
  p.codes = static_cast<uint2*>(codes);
  p.scales = scales;
  p.Kr = (int)(K / kWorld);
  p.vec = (int)(N / 8);
  p.kb = (int)blocks_of(p.Kr);
  p.nb = (int)blocks_of(N);
  const dim3 grid((unsigned)(experts * kWorld * p.kb * p.nb));
  return launch_overlapped(scale == kFp8F32 ? quantize_weight_kernel<false> : quantize_weight_kernel<true>, grid, kThreads, 0,
                           static_cast<cudaStream_t>(stream), p);
}

}  // namespace

extern "C" int gemm_rs_fp8_weight_bytes(int64_t experts, int64_t N, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  return weight_bytes(kFp8F32, experts, N, K, code_bytes, scale_bytes);
}
extern "C" int gemm_rs_fp8_weight_bytes_e8m0(int64_t experts, int64_t N, int64_t K, size_t* code_bytes,
                                             size_t* scale_bytes) {
  return weight_bytes(kFp8E8m0, experts, N, K, code_bytes, scale_bytes);
}
extern "C" int gemm_rs_fp8_quantize(int64_t experts, int64_t N, int64_t K, const void* W, void* codes, void* scales,
                                    void* stream) {
  return quantize(kFp8F32, experts, N, K, W, codes, scales, stream);
}
extern "C" int gemm_rs_fp8_quantize_e8m0(int64_t experts, int64_t N, int64_t K, const void* W, void* codes, void* scales,
                                         void* stream) {
  return quantize(kFp8E8m0, experts, N, K, W, codes, scales, stream);
}

extern "C" int gemm_rs_fp8_checkpoint_bytes(int64_t M, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  const int rc = check_shape(M, 0, K);
  if (rc) return rc;
  if (code_bytes) *code_bytes = (size_t)kWorld * padded_rows(M, 1) * fp8_pitch(K / kWorld);
  if (scale_bytes) *scale_bytes = token_scale_bytes(padded_rows(M, 1), kWorld, K / kWorld);
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_fp8_workspace(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  const int rc = check_shape(M, N, K);
  if (rc) return rc;
  const size_t f = forward_places(M, N, K).total, b = backward_places(M, N).total;
  if (bytes) *bytes = f > b ? f : b;
  return GEMM_RS_OK;
}

namespace {

int forward(Fp8Scale scale, int64_t M, int64_t N, int64_t K, const void* A, const void* codes, const void* scales,
            void* ck_codes, void* ck_scales, void* out, void* workspace, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((ck_codes == nullptr) != (ck_scales == nullptr) && M > 0 && K > 0) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {A, codes, (const void*)ck_codes, (const void*)ck_scales, (const void*)out,
                        (const void*)workspace})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (misaligned_scales(scale, scales)) return GEMM_RS_ERR_MISALIGNED;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  if (M == 0 || K == 0) {  // nothing to multiply
    rc = clear(workspace, sizeof(uint32_t), st);
    return rc ? rc : clear(out, (size_t)M * N * 2, st);
  }
  if (!A || (N > 0 && (!codes || !scales || !out))) return GEMM_RS_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const Places w = forward_places(M, N, K);
  Fp8Quantize q;
  q.scale = scale;
  q.x = A;
  q.planes = kWorld;
  q.cols = K / kWorld;
  q.rows.M = M;
  q.row_codes = at<void>(workspace, w.row_codes);
  q.row_scales = at<void>(workspace, w.row_scales);
  q.token_codes = ck_codes;
  q.token_scales = ck_scales;
  q.status = at<uint32_t>(workspace, 0);
  rc = fp8_quantize_rows(q, st);
  if (rc || N == 0) return rc;
  if (fp8_few_serves(kFp8Forward, q.rows, N, K / kWorld, false, sms)) {
    Fp8Few f;
    f.scale = scale;
    f.kind = kFp8Forward;
    f.N = N;
    f.Kr = K / kWorld;
    f.rows = q.rows;
    f.a = q.row_codes;
    f.a_scale = q.row_scales;
    f.b = codes;
    f.b_scale = scales;
    f.out = out;
    f.status = q.status;
    return fp8_few(f, st);
  }
  Fp8Product p;
  p.scale = scale;
  p.kind = kFp8Forward;
  p.N = N;
  p.Kr = K / kWorld;
  p.rows = q.rows;
  p.a = q.row_codes;
  p.a_scale = q.row_scales;
  p.b = codes;
  p.b_scale = scales;
  p.out = out;
  p.status = q.status;
  p.parts = parts_of(M, N, K);
  if (p.parts == 1) return fp8_product(p, st);
  p.out = at<void>(workspace, w.parts);
  p.out_f32 = true;
  rc = fp8_product(p, st);
  if (rc) return rc;
  SumParams s;
  s.parts = at<float>(workspace, w.parts);
  s.out = static_cast<uint4*>(out);
  s.vec = M * N / 8;
  s.count = p.parts;
  return launch_overlapped(sum_parts_kernel, dim3((unsigned)((s.vec + kThreads - 1) / kThreads)), kThreads, 0, st, s);
}

int backward(Fp8Scale scale, int64_t M, int64_t N, int64_t K, const void* dY, const void* codes, const void* scales,
             const void* ck_codes, const void* ck_scales, void* dA, void* dW, void* workspace, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (const void* q : {dY, codes, ck_codes, ck_scales, (const void*)dA, (const void*)dW, (const void*)workspace})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (misaligned_scales(scale, scales)) return GEMM_RS_ERR_MISALIGNED;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  if (M == 0 || N == 0 || K == 0) {  // an empty contraction
    rc = clear(workspace, sizeof(uint32_t), st);
    if (!rc && dA) rc = clear(dA, (size_t)M * K * 2, st);
    if (!rc && dW) rc = clear(dW, (size_t)K * N * 2, st);
    return rc;
  }
  if (!dA && !dW) return clear(workspace, sizeof(uint32_t), st);
  if (!dY || (dA && (!codes || !scales)) || (dW && (!ck_codes || !ck_scales))) return GEMM_RS_ERR_INVALID_ARG;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const Places w = backward_places(M, N);
  Fp8Quantize q;
  q.scale = scale;
  q.x = dY;
  q.planes = 1;
  q.cols = N;
  q.rows.M = M;
  if (dA) {
    q.row_codes = at<void>(workspace, w.row_codes);
    q.row_scales = at<void>(workspace, w.row_scales);
  }
  if (dW) {
    q.token_codes = at<void>(workspace, w.token_codes);
    q.token_scales = at<void>(workspace, w.token_scales);
  }
  q.status = at<uint32_t>(workspace, 0);
  const bool few = dA && fp8_few_serves(kFp8InputGrad, q.rows, N, K / kWorld, dW != nullptr, sms);
  rc = fp8_quantize_rows(q, st);
  if (rc) return rc;
  Fp8Product p;
  p.scale = scale;
  p.N = N;
  p.Kr = K / kWorld;
  p.rows = q.rows;
  p.status = q.status;
  Fp8Product g = p;
  if (few) {
    Fp8Few f;
    f.scale = scale;
    f.kind = kFp8InputGrad;
    f.N = N;
    f.Kr = K / kWorld;
    f.rows = q.rows;
    f.a = q.row_codes;
    f.a_scale = q.row_scales;
    f.b = codes;
    f.b_scale = scales;
    f.out = dA;
    f.status = q.status;
    rc = fp8_few(f, st);
    if (rc) return rc;
  } else if (dA) {
    p.kind = kFp8InputGrad;
    p.a = q.row_codes;
    p.a_scale = q.row_scales;
    p.b = codes;
    p.b_scale = scales;
    p.out = dA;
  }
  if (dW) {
    g.kind = kFp8WeightGrad;
    g.a = ck_codes;
    g.a_scale = ck_scales;
    g.b = q.token_codes;
    g.b_scale = q.token_scales;
    g.out = dW;
  }
  if (dA && dW && !few) return fp8_products(p, g, st);
  if (dA && !few) return fp8_product(p, st);
  if (dW) return fp8_product(g, st);
  return rc;
}

}  // namespace

extern "C" int gemm_rs_fp8_forward(int64_t M, int64_t N, int64_t K, const void* A, const void* codes, const void* scales,
                                   void* ck_codes, void* ck_scales, void* out, void* workspace, void* stream) {
  return forward(kFp8F32, M, N, K, A, codes, scales, ck_codes, ck_scales, out, workspace, stream);
}
extern "C" int gemm_rs_fp8_forward_e8m0(int64_t M, int64_t N, int64_t K, const void* A, const void* codes,
                                        const void* scales, void* ck_codes, void* ck_scales, void* out, void* workspace,
                                        void* stream) {
  return forward(kFp8E8m0, M, N, K, A, codes, scales, ck_codes, ck_scales, out, workspace, stream);
}
extern "C" int gemm_rs_fp8_backward(int64_t M, int64_t N, int64_t K, const void* dY, const void* codes,
                                    const void* scales, const void* ck_codes, const void* ck_scales, void* dA, void* dW,
                                    void* workspace, void* stream) {
  return backward(kFp8F32, M, N, K, dY, codes, scales, ck_codes, ck_scales, dA, dW, workspace, stream);
}
extern "C" int gemm_rs_fp8_backward_e8m0(int64_t M, int64_t N, int64_t K, const void* dY, const void* codes,
                                         const void* scales, const void* ck_codes, const void* ck_scales, void* dA,
                                         void* dW, void* workspace, void* stream) {
  return backward(kFp8E8m0, M, N, K, dY, codes, scales, ck_codes, ck_scales, dA, dW, workspace, stream);
}

extern "C" int gemm_rs_fp8_status(const void* workspace, void* stream) {
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, workspace, sizeof(word), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_RS_ERR_CUDA;
  }
  return word ? GEMM_RS_ERR_TIMEOUT : GEMM_RS_OK;
}
