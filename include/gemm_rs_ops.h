/*
 * gemm_rs_ops.h -- C ABI of the operators around the row-parallel layer of
 * gemm_rs.h (same library, same status codes, same conventions).
 *
 *   norm   the norms after and before a block, fused with the block's gate and
 *          residual scale, forward and backward
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
  int64_t M, D;       /* M >= 0; D a positive multiple of 8, at most 16384 */
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

#ifdef __cplusplus
}
#endif

#endif /* GEMM_RS_OPS_H */
