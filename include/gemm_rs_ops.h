/*
 * gemm_rs_ops.h -- C ABI of the operators around the row-parallel layer of
 * gemm_rs.h (same library, same status codes, same conventions).
 *
 *   norm   the norms after and before a block, fused with the block's gate and
 *          residual scale, forward and backward
 *   act8   the layer's input kept in 8 bits between the forward and the
 *          backward pass, and the layer's backward pass from it (gemm_rs_bwd_*)
 *   w4     the layer for 1 to 32 tokens, with 4-bit weights and group scales
 *   fp8    the layer in 8-bit floating point with a scale for each block of 128,
 *          forward and backward
 *   moe    routing to experts, and their layer in fp8 with a weight for each
 *          token and expert, forward and backward
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

/* -------------------------------------------------------------------- fp8
 * The row-parallel layer in e4m3 (4 bits of exponent, 3 of mantissa, largest
 * 448) with a scale for each block of 128.  A block's scale is
 * max(largest magnitude, 2^-100) * fp32(1/448), rounded to fp32; a code is the
 * element times the scale's fp32 reciprocal, rounded to fp32, then to e4m3, to
 * nearest even.  A block with an infinity or a NaN has the scale NaN and NaN codes,
 * and so makes NaN of every output that it takes part in.  In the products
 *
 *   out    = sum_r A_r W_r     A in 1 x 128 blocks along K/8, W in 128 x 128
 *   dA_r   = dY W_r^T          dY in 1 x 128 blocks along N, W as above
 *   dW_r   = A_r^T dY          A and dY in blocks of 128 tokens for each column
 *
 * the codes of a step of 128 inner elements are multiplied and summed on the
 * tensor cores in fp32, scaled by the product of the two scales, and added up
 * in fp32 (where the product of two scales is no normal number of fp32, the step loses
 * bits, or is infinite or NaN); outputs are rounded to bf16 once.  The same call gives the same bits; with
 * other rows beside it, or for dA without dW, a sum may run in another order.
 *
 * Weights: codes [experts][8][ceil(N/128)][K/8][128] e4m3 (128 columns of W at a
 * time; zero behind the last column) and scales [experts][8][ceil(K/8/128)]
 * [ceil(N/128)] fp32.  Codes and scales made elsewhere in this layout serve as
 * well.  experts is 1 for the layer itself.
 *
 * The entries whose names end in _e8m0 are the same in a form that large products
 * take 0.6 to 0.8 of the time in, for some accuracy: every block's scale, of weights, inputs and
 * gradients alike, is a power of two, 2^e with the least e >= -126 such that the
 * block's largest magnitude is at most 448 * 2^e; codes are the elements over 2^e,
 * and the tensor cores apply the scales, so that the whole contraction is summed in
 * their fp32 (which may truncate where it aligns addends).  The weights' scales are
 * bytes, e + 127, 255 for NaN.  Inputs with one entry in 20 eight times as large are rounded by
 * 2.7% of their norm in this form, and by 2.1% in the other.  A checkpoint serves the form that wrote it.
 *
 * N % 8 == 0, K % 64 == 0, any M; 0 allowed. */
#define GEMM_RS_FP8_MAX_EXPERTS 256
int gemm_rs_fp8_weight_bytes(int64_t experts, int64_t N, int64_t K, size_t* code_bytes,
                             size_t* scale_bytes); /* host only */
/* Codes and scales of W [experts][8][K/8][N] bf16. */
int gemm_rs_fp8_quantize(int64_t experts, int64_t N, int64_t K, const void* W, void* codes,
                         void* scales, void* stream);
int gemm_rs_fp8_weight_bytes_e8m0(int64_t experts, int64_t N, int64_t K, size_t* code_bytes,
                                  size_t* scale_bytes); /* host only */
int gemm_rs_fp8_quantize_e8m0(int64_t experts, int64_t N, int64_t K, const void* W, void* codes,
                              void* scales, void* stream);
/* What the backward pass keeps of A: its codes in blocks of 128 tokens and their
 * scales, contents private to this library.  Either form's. */
int gemm_rs_fp8_checkpoint_bytes(int64_t M, int64_t K, size_t* code_bytes,
                                 size_t* scale_bytes); /* host only */
/* Bytes of workspace of either pass in either form (host only).  It needs no initialisation. */
int gemm_rs_fp8_workspace(int64_t M, int64_t N, int64_t K, size_t* bytes);
/* A [8][M][K/8], out [M][N] bf16; codes and scales of the weight.  ck_codes and
 * ck_scales (both or neither) take what the backward pass needs. */
int gemm_rs_fp8_forward(int64_t M, int64_t N, int64_t K, const void* A, const void* codes,
                        const void* scales, void* ck_codes, void* ck_scales, void* out,
                        void* workspace, void* stream);
/* dY [M][N], dA [8][M][K/8], dW [8][K/8][N] bf16.  dA or dW may be NULL when it is
 * not needed (the weight, or the checkpoint, may then be NULL too). */
int gemm_rs_fp8_backward(int64_t M, int64_t N, int64_t K, const void* dY, const void* codes,
                         const void* scales, const void* ck_codes, const void* ck_scales,
                         void* dA, void* dW, void* workspace, void* stream);
int gemm_rs_fp8_forward_e8m0(int64_t M, int64_t N, int64_t K, const void* A, const void* codes,
                             const void* scales, void* ck_codes, void* ck_scales, void* out,
                             void* workspace, void* stream);
int gemm_rs_fp8_backward_e8m0(int64_t M, int64_t N, int64_t K, const void* dY, const void* codes,
                              const void* scales, const void* ck_codes, const void* ck_scales,
                              void* dA, void* dW, void* workspace, void* stream);
/* Device-side waits are bounded (2 s).  The status of the last call with this
 * workspace: synchronises `stream`; GEMM_RS_OK, GEMM_RS_ERR_TIMEOUT (a wait gave
 * up, the outputs are incomplete) or GEMM_RS_ERR_CUDA. */
int gemm_rs_fp8_status(const void* workspace, void* stream);

/* -------------------------------------------------------------------- moe
 * Routing of T tokens to top_k of E experts, from logits [T][E] (fp32 or bf16):
 *
 *   score  = softmax over the E experts, or sigmoid of each
 *   choice = score + bias[e]                            (bias [E] fp32 or NULL)
 *   the experts lie in `groups` groups of E/groups; the top_groups groups with the
 *   largest sums of their two largest choices stay (of one, if groups are of one; the
 *   sum of inf and -inf counts as inf)
 *   ids    = the top_k experts of those groups with the largest choice, in
 *            descending order, the lower index first where two are equal
 *   weight = scale * score / (sum of the chosen scores, if renormalize)
 *
 * ids do not depend on rounding: values that fp32 cannot tell apart are compared in
 * 64 bits.  Without a bias experts of a group are compared by their logits.  A token
 * whose mask byte is 0 (mask [T] or NULL) gets ids -1 and weights 0.  A logit of
 * -inf has the score 0; weights are 0 where every chosen score is.  Logits of +inf
 * share a softmax equally and leave nothing to the others.  A NaN counts as the lowest
 * logit, of score 0, for the choice, and makes the token's weights and gradient NaN.
 *
 * The token-expert pairs (pair t * top_k + j) are put in the order of their
 * experts, then of the pairs: rows [T][top_k] is each pair's place (-1 without an
 * expert), pairs [T * top_k] the pair at each place, offsets [E + 1] the first
 * place of each expert and, last, the number of pairs with an expert; pairs behind
 * that one is left as it was.  ids, rows, pairs, offsets int32, weights fp32. */
#define GEMM_RS_MOE_MAX_TOP_K 16
typedef struct gemm_rs_route_desc {
  int64_t T, E;       /* T >= 0, at most 2^22; E from 1 to GEMM_RS_FP8_MAX_EXPERTS */
  int32_t top_k;      /* 1 to GEMM_RS_MOE_MAX_TOP_K, at most top_groups * E/groups */
  int32_t logits_bf16; /* 0: fp32 */
  int32_t score;      /* 0 softmax, 1 sigmoid */
  int32_t groups;     /* a divisor of E, at most 32; 1: none */
  int32_t top_groups; /* 1 to groups */
  int32_t renormalize;
  float scale;
} gemm_rs_route_desc;

int gemm_rs_moe_route(const gemm_rs_route_desc* d, const void* logits, const void* bias,
                      const void* mask, void* ids, void* weights, void* rows, void* pairs,
                      void* offsets, void* stream);
/* rows, pairs and offsets for ids from elsewhere; an id outside 0..E-1 is no expert. */
int gemm_rs_moe_arrange(int64_t T, int64_t E, int64_t top_k, const void* ids, void* rows,
                        void* pairs, void* offsets, void* stream);
/* dlogits [T][E] (of the logits' type) for dweights [T][top_k] fp32; ids as chosen.  The
 * choice itself and the bias have no gradient. */
int gemm_rs_moe_route_backward(const gemm_rs_route_desc* d, const void* dweights,
                               const void* logits, const void* ids, void* dlogits, void* stream);

/* The experts' row-parallel layer in fp8 (see there for blocks and rounding), for
 * pairs in the order above: A [8][T * top_k][K/8] bf16 holds each pair's input at
 * its place, codes and scales are the experts' weights, and
 *
 *   y[row]      = sum_r A_r[row] W[expert of row]_r              fp32
 *   out[t]      = sum_j weights[t][j] y[rows[t][j]]              bf16, one rounding
 *   dy[row]     = weights[t][j] dout[t], rounded to fp32         pair (t, j) at row
 *   dA_r[row]   = dy[row] W[e]_r^T            dweights[t][j] = sum_n dout[t][n] y[row][n]
 *   dW[e]_r     = A_r[rows of e]^T dy[rows of e]
 *
 * with A and dy in blocks along their rows for y and dA, and in blocks of 128 rows of
 * an expert, from its first, for dW.  Rows behind the last pair with an expert are
 * not read and, in dA, left as they were.  An expert without rows gets dW = 0.
 * Places and pairs outside the tensors are passed over, in rows, pairs and offsets
 * that were not made by the calls above. */
typedef struct gemm_rs_moe_desc {
  int64_t T, E, top_k; /* limits as above, top_k may exceed E */
  int64_t N, K;        /* N % 8 == 0, K % 64 == 0 */
} gemm_rs_moe_desc;

/* What the backward pass keeps: codes and scales of A, private to this library, and
 * y [T * top_k][N] fp32 (host only). */
int gemm_rs_moe_checkpoint_bytes(const gemm_rs_moe_desc* d, size_t* code_bytes,
                                 size_t* scale_bytes, size_t* y_bytes);
/* Bytes of workspace of either pass (host only).  It needs no initialisation;
 * gemm_rs_fp8_status reads the status of the last call with it. */
int gemm_rs_moe_workspace(const gemm_rs_moe_desc* d, size_t* bytes);
/* ck_codes, ck_scales and ck_y (all or none) take what the backward pass needs. */
int gemm_rs_moe_forward(const gemm_rs_moe_desc* d, const void* A, const void* codes,
                        const void* scales, const void* weights, const void* rows,
                        const void* offsets, void* ck_codes, void* ck_scales, void* ck_y,
                        void* out, void* workspace, void* stream);
/* dA, dW or dweights may be NULL when it is not needed, and then what only it needs. */
int gemm_rs_moe_backward(const gemm_rs_moe_desc* d, const void* dout, const void* codes,
                         const void* scales, const void* weights, const void* rows,
                         const void* pairs, const void* offsets, const void* ck_codes,
                         const void* ck_scales, const void* ck_y, void* dA, void* dW,
                         void* dweights, void* workspace, void* stream);
/* With scales that are powers of two (see fp8). */
int gemm_rs_moe_forward_e8m0(const gemm_rs_moe_desc* d, const void* A, const void* codes,
                             const void* scales, const void* weights, const void* rows,
                             const void* offsets, void* ck_codes, void* ck_scales, void* ck_y,
                             void* out, void* workspace, void* stream);
int gemm_rs_moe_backward_e8m0(const gemm_rs_moe_desc* d, const void* dout, const void* codes,
                              const void* scales, const void* weights, const void* rows,
                              const void* pairs, const void* offsets, const void* ck_codes,
                              const void* ck_scales, const void* ck_y, void* dA, void* dW,
                              void* dweights, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RS_OPS_H */
