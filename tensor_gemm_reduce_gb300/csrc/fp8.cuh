// fp8.cuh -- shared by the operators in 8-bit floating point (fp8.cu, moe.cu):
// block sizes and layouts, the quantising kernels and the tensor-core product.
#pragma once
#include "ops_common.cuh"
#include "schedule.h"

namespace grs {

constexpr int kBlk = 128;          // elements that share a scale along an axis
constexpr int kMaxExperts = 256;   // of one weight
constexpr size_t kFp8Status = 256; // bytes in front of a workspace: word 0 is the last call's status

inline int64_t blocks_of(int64_t n) { return (n + kBlk - 1) / kBlk; }
inline int64_t fp8_pitch(int64_t n) { return (n + 15) / 16 * 16; }    // bytes between rows of codes: TMA strides
inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }
// Sizes whose tile and block indices fit 32 bits (experts: 1 to kMaxExperts).
int fp8_check_sizes(int64_t M, int64_t experts, int64_t N, int64_t K);
// Rows of token-blocked codes: every expert's tokens start at a multiple of 128.
inline int64_t padded_rows(int64_t M, int64_t experts) {
  return (blocks_of(M) + (experts > 1 ? experts - 1 : 0)) * kBlk;
}

// The rows of an activation: tokens, or token-expert pairs in the order of their experts.
struct Fp8Rows {
  int64_t M = 0;                  // rows that the tensors hold
  int experts = 1;
  const int* offsets = nullptr;   // [experts + 1] first row of each expert, device; null: one expert, all M rows
  // a row's source where the rows are gathered from tokens: pair -> row / top_k, times weight[pair]
  const int* pairs = nullptr;     // [M]
  const float* weights = nullptr; // [tokens * top_k]
  int top_k = 1;
};

// What a block's scale is: fp32 of its largest magnitude over 448, or the least power of two that
// holds it (a byte, its exponent).
enum Fp8Scale { kFp8F32 = 0, kFp8E8m0 = 1 };

// e4m3 codes of x [planes][M][cols] bf16.  By rows: 1 x 128 blocks along cols, codes
// [planes][M][pitch]; a scale for each of the planes * ceil(cols/128) blocks and row.  By tokens:
// blocks of 128 rows of an expert, codes [planes][padded rows][pitch]; a scale for each block, plane
// and column.  Bytes lie in words for four blocks.  Either may be absent.  status (if not null) is
// set to zero.
struct Fp8Quantize {
  const void* x;
  int planes;
  int64_t cols;
  Fp8Rows rows;
  Fp8Scale scale;
  void* row_codes = nullptr;
  void* row_scales = nullptr;    // fp32 [blocks][row_scale_pitch(M)], bytes [ceil(blocks / 4)][row_scale_pitch(M)][4]
  void* token_codes = nullptr;
  void* token_scales = nullptr;  // fp32 [blocks][planes][pitch], bytes [ceil(blocks / 4)][planes][pitch][4]
  uint32_t* status = nullptr;
};
int fp8_quantize_rows(const Fp8Quantize& q, cudaStream_t stream);

// The first row of expert e (the end of e - 1), whatever the caller's offsets hold, no row
// outside the tensors.
__device__ __forceinline__ int expert_row(const int* offsets, int e, int M) {
  int row;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(row) : "l"(offsets + e) : "memory");
  return row < 0 ? 0 : row < M ? row : M;
}

inline int64_t row_scale_pitch(int64_t M) { return (M + 3) / 4 * 4; }
// Bytes of the scales of either kind: fp32's are the more.
inline size_t row_scale_bytes(int64_t M, int64_t blocks) { return (size_t)blocks * row_scale_pitch(M) * 4; }
inline size_t token_scale_bytes(int64_t rows, int planes, int64_t cols) {
  return (size_t)(rows / kBlk) * planes * fp8_pitch(cols) * 4;
}

enum Fp8Kind { kFp8Forward = 0, kFp8InputGrad = 1, kFp8WeightGrad = 2 };

// One product on the tensor cores, for each expert's rows:
//   forward      out[m][n]      = sum_r sum_k a[r][m][k] w[e][r][k][n]
//   input grad   out[r][m][k]   = sum_n a[m][n] w[e][r][k][n]
//   weight grad  out[e][r][k][n] = sum_m a[r][m][k] b[m][n]   over the expert's padded rows
struct Fp8Product {
  Fp8Kind kind;
  Fp8Scale scale;
  int64_t N, Kr;
  Fp8Rows rows;
  const void* a;          // codes: forward [8][M][pitch(Kr)], input grad [M][pitch(N)], weight grad [8][padded][pitch(Kr)]
  const void* a_scale;    // as fp8_quantize_rows lays them out
  const void* b;          // codes: the weight [e][8][ceil(N/128)][Kr][128]; weight grad [padded][pitch(N)]
  const void* b_scale;    // the weight's [e][8][ceil(Kr/128)][ceil(N/128)]; weight grad: as a's
  void* out;
  bool out_f32 = false;   // forward only
  int parts = 1;          // forward of one weight, into fp32: [parts][M][N], a run of the contraction each
  uint32_t* status;
};
int fp8_product_f32(const Fp8Product& p, cudaStream_t stream);
int fp8_product_e8m0(const Fp8Product& p, cudaStream_t stream);
inline int fp8_product(const Fp8Product& p, cudaStream_t stream) {
  return p.scale == kFp8F32 ? fp8_product_f32(p, stream) : fp8_product_e8m0(p, stream);
}
// dA and dW of the same rows in one launch.
int fp8_products_f32(const Fp8Product& input, const Fp8Product& weight, cudaStream_t stream);
int fp8_products_e8m0(const Fp8Product& input, const Fp8Product& weight, cudaStream_t stream);
inline int fp8_products(const Fp8Product& input, const Fp8Product& weight, cudaStream_t stream) {
  return input.scale == kFp8F32 ? fp8_products_f32(input, weight, stream) : fp8_products_e8m0(input, weight, stream);
}

// The forward product or dA for few rows, which reads each weight once: out [M][N] or
// [8][M][Kr], or for experts' forward out [tokens][N] = sum_j weights[t][j] y[place[t][j]], y also
// stored where it is wanted.  The launch before it on the stream is the quantisation of its rows.
constexpr int kFewRows = 128;
struct Fp8Few {
  Fp8Kind kind;
  Fp8Scale scale;
  int64_t N, Kr;
  Fp8Rows rows;
  const void* a;
  const void* a_scale;
  const void* b;
  const void* b_scale;
  void* out;
  int64_t tokens = 0;             // experts' forward: of out, top_k rows each
  const float* weights = nullptr; // [tokens][top_k]
  const int* place = nullptr;     // [tokens][top_k]
  float* y = nullptr;             // [M][N] or null
  uint32_t* status;
};
// Whether fp8_few takes less time than fp8_product; with_weight_grad: dA beside which dW is wanted too,
// which fp8_products would multiply in the same launch.
bool fp8_few_serves(Fp8Kind kind, const Fp8Rows& rows, int64_t N, int64_t Kr, bool with_weight_grad, int sms);
int fp8_few(const Fp8Few& p, cudaStream_t stream);

}  // namespace grs
