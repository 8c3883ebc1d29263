/*
 * gemm_rs_ops.h -- C ABI of the operators around the row-parallel layer of
 * gemm_rs.h (same library, same status codes, same conventions).
 *
 *   norm   the norms after and before a block, fused with the block's gate and
 *          residual scale, forward and backward
 *   act8   the layer's input kept in 8 bits between the forward and the
 *          backward pass, and the layer's backward pass from it (gemm_rs_bwd_*)
 *   w4     the layer for 1 to 32 tokens, with 4-bit weights and group scales
 *
 * Every device buffer and the CUDA stream belong to the caller; nothing here
 * allocates device memory or synchronises unless a comment says so.  Buffers
 * are contiguous, row-major and 16-byte aligned; outputs do not overlap inputs.
 * Arguments are checked before any CUDA call.  Calls only enqueue work on
 * `stream` (a cudaStream_t; NULL = legacy default).  No C++ exception and no
 * abort crosses this boundary.  Pointers are device pointers unless a comment
 * says "host".
 */
#ifndef GEMM_RS_OPS_H
#define GEMM_RS_OPS_H

#include "gemm_rs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------- norm
 * x: residual stream [M][D], y: the block's output [M][D] (the reduced output
 * of the row-parallel layer), w_post, w_pre: [D], gate: [gate_rows][D] or
 * NULL, all bf16.  Gate row i serves rows [i*M/gate_rows, (i+1)*M/gate_rows):
 * 1 row is a gate per channel, M rows one per element, the batch size one per
 * sequence.
 *
 *   p = 1 / sqrt(mean(y^2) + eps)              u = y * p * w_post
 *   r = x + scale * gate * u                   (gate = 1 without one)
 *   q = 1 / sqrt(mean(r^2) + eps)              h = r * q * w_pre
 *
 * r is the residual stream after the block, h the next block's input.  All
 * arithmetic is fp32; r and h are rounded to bf16 once, and h is computed
 * from the unrounded r.
 */
typedef struct gemm_rs_norm_desc {
  int64_t M, D;       /* M >= 0; D a positive multiple of 8, at most 16384; M * D <= 2^34 */
  int64_t gate_rows;  /* 0: no gate; else a positive divisor of M (any, if M = 0) */
  float scale;        /* residual scale of the block's branch */
  float eps;          /* >= 0; not read by the backward pass */
} gemm_rs_norm_desc;

#define GEMM_RS_NORM_MAX_D 16384

/* Outputs r, h: [M][D] bf16; stats: [2][M] fp32, p then q (may be NULL when no
 * backward pass follows). */
int gemm_rs_norm_forward(const gemm_rs_norm_desc* d, const void* x, const void* y,
                         const void* gate, const void* w_post, const void* w_pre, void* r,
                         void* h, void* stats, void* stream);

/* Bytes of workspace of the backward pass (host only). */
int gemm_rs_norm_workspace(const gemm_rs_norm_desc* d, size_t* bytes);

/* Gradients for dr, dh: [M][D] bf16 (with respect to r and h); x, y, gate,
 * w_post, w_pre as in the forward pass and stats as it wrote them.  Outputs dx,
 * dy: [M][D], dgate: [gate_rows][D] (NULL without a gate), dw_post, dw_pre:
 * [D], all bf16, overwritten.  Sums over rows are fp32 in a fixed order: the
 * same call gives the same bits.  With M = 0 the weight gradients are zero.
 * The workspace needs no initialisation. */
int gemm_rs_norm_backward(const gemm_rs_norm_desc* d, const void* dr, const void* dh,
                          const void* x, const void* y, const void* gate, const void* w_post,
                          const void* w_pre, const void* stats, void* dx, void* dy, void* dgate,
                          void* dw_post, void* dw_pre, void* workspace, void* stream);

/* ------------------------------------------------------------------- act8
 * An 8-bit checkpoint of A [8][M][K/8] bf16.  32 consecutive elements of a row
 * (fewer at its end) share a power of two: 2^e with the least e >= -126 such
 * that the largest magnitude is at most 127 * 2^e; each element is kept as
 * round(a / 2^e) (to nearest even, at most 7 bits and a sign), so the restored
 * value is exact in bf16.  (Magnitudes that would round to 2^128 keep the
 * largest code below it.)  A group with an infinity or a NaN is restored as
 * NaN throughout.
 *
 * codes: [8][M][pitch] bytes, scales: [8][M][pitch/32] bytes, pitch = K/8
 * rounded up to 128; the contents of both are private to this library.
 * Shapes as in gemm_rs.h: M % 8 == 0, K % 64 == 0; 0 allowed.
 */
int gemm_rs_act8_layout(int64_t M, int64_t K, int64_t* pitch, size_t* code_bytes,
                        size_t* scale_bytes); /* host only */
int gemm_rs_act8_save(int64_t M, int64_t K, const void* A, void* codes, void* scales,
                      void* stream);
int gemm_rs_act8_restore(int64_t M, int64_t K, const void* codes, const void* scales, void* A,
                         void* stream);

/* Backward pass of the row-parallel layer out = sum_r A_r W_r, with A from a
 * checkpoint: for the output's gradient dY [M][N],
 *   dA_r = dY W_r^T   [8][M][K/8]          dW_r = A_r^T dY   [8][K/8][N]
 * bf16 in and out, fp32 accumulation, one rounding.  dA or dW may be NULL when
 * it is not needed (W, or codes and scales, may then be NULL too). */
typedef struct gemm_rs_bwd_plan_s* gemm_rs_bwd_t;

/* timeout_ns: bound on every device-side wait; 0 = 2 s (a run that gives up takes
 * about 10 ms more to end).  Shapes are checked before any CUDA call.  N % 8 == 0,
 * the others as above.  The plan is for the device that is current here. */
int gemm_rs_bwd_create(int64_t M, int64_t N, int64_t K, uint64_t timeout_ns, gemm_rs_bwd_t* plan,
                       size_t* workspace_bytes);
/* The workspace needs no initialisation, and plans that follow one another on a
 * stream may share one.  gemm_rs_bwd_status reads it, so it stays allocated until
 * the last call of that for this run.  A plan serves one stream at a time. */
int gemm_rs_bwd_run(gemm_rs_bwd_t plan, const void* dY, const void* W, const void* codes,
                    const void* scales, void* dA, void* dW, void* workspace, void* stream);
/* Status of the last run in the plan's last workspace, which it reads and does not
 * change.  Synchronises `stream`; GEMM_RS_OK, GEMM_RS_ERR_TIMEOUT (a device-side
 * wait gave up, the outputs are incomplete) or GEMM_RS_ERR_CUDA. */
int gemm_rs_bwd_status(gemm_rs_bwd_t plan, void* stream);
int gemm_rs_bwd_destroy(gemm_rs_bwd_t plan);

/* --------------------------------------------------------------------- w4
 * The row-parallel layer for few tokens with 4-bit weights.  `group`
 * consecutive inner elements of a rank's shard (32, 64 or 128; fewer at its
 * end) share, for each column, a scale and optionally a zero point:
 *
 *   out[m][n] = sum_r sum_k x[r][m][k] (code[r][k][n] - zero[r][k/group][n]) scale[r][k/group][n]
 *
 * x [8][M][K/8] bf16, M from 0 to 32; codes [8][K/8][N] bytes 0..15 (the low
 * four bits count); scales [8][ceil(K/8/group)][N] bf16; zeros of that shape,
 * bytes 0..127 (the low seven bits count), or NULL for 8 everywhere; out [M][N]
 * bf16.  Products are summed in fp32 in a fixed order and rounded once.
 * N % 8 == 0, at most 2^19; K % 64 == 0.
 *
 * The weights are packed once into one buffer, whose contents are private to
 * this library; codes, scales and zeros are not needed after that. */
int gemm_rs_w4_bytes(int64_t N, int64_t K, int group, int has_zeros,
                     size_t* weight_bytes); /* host only */
/* Symmetric codes of W [8][K/8][N] bf16, rounded to nearest: scale =
 * bf16(largest magnitude of the group / 7), code = 8 + round(w / scale) in
 * 0..15; a group with an infinity or a NaN gets the scale NaN. */
int gemm_rs_w4_quantize(int64_t N, int64_t K, int group, const void* W, void* codes, void* scales,
                        void* stream);
int gemm_rs_w4_pack(int64_t N, int64_t K, int group, const void* codes, const void* scales,
                    const void* zeros, void* weight, void* stream);
/* Needs no workspace. */
int gemm_rs_w4_run(int64_t M, int64_t N, int64_t K, int group, int has_zeros, const void* x,
                   const void* weight, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RS_OPS_H */
