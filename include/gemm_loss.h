/*
 * gemm_loss.h -- softmax losses over the logits of a vocabulary product (gfx950).
 *
 * The logits z = x . w^T of T rows over V vocabulary entries are not kept: they
 * are reduced where the matrix cores produce them, in pieces of the vocabulary.
 *
 *   x [T,H] bf16/fp16      w [V,H] (GEMM_B_NK) or [H,V] (GEMM_B_KN), same type
 *   lse_t = log sum_v exp(z_tv / tau)                       p_tv = exp(z_tv / tau - lse_t)
 *
 * GEMM_LOSS_XENT (cross entropy, tau = 1), target y_t:
 *   loss_t = lse_t - z_t[y_t] + zeta lse_t^2
 *   dz_tv  = g_t ((1 + 2 zeta lse_t) p_tv - [v = y_t])
 * GEMM_LOSS_DISTILL (a teacher's top logits), entries i_tk with teacher logits s_tk:
 *   q_t    = softmax over the row's entries of s_t / tau
 *   loss_t = tau^2 sum_k q_tk (log q_tk - z_t[i_tk] / tau + lse_t)
 *   dz_tv  = g_t tau (p_tv - sum_{k: i_tk = v} q_tk)
 * and in both  dx = dz . w,  dw = dz^T . x  (stored as w is).
 *
 * Rows without a target have loss 0 and no gradient: y_t = ignore_index; or no
 * entry with i_tk >= 0 and a teacher logit above -infinity.  Single entries
 * i_tk < 0 are padding; what their teacher logits hold does not matter.  The
 * same entry named twice counts twice.  A target or entry >= V (or a negative
 * target other than ignore_index) makes the row's loss NaN, and so its
 * gradient: nothing is read out of range.  lse is written for every row.
 * x must be finite in rows without a target too when dw is computed (their
 * gradient is zero, and zero times infinity is not).
 *
 * Arithmetic: logits, maxima, sums of exponentials and losses in fp32.  The
 * backward pass computes the logits again, rounds dz to the operands' type (up to
 * 64 rows: to the sum of two such values) once
 * (fp16: after scaling by a power of two that brings the largest row factor to
 * at most 2^14, divided out of dx and dw: besides its rounding an entry of any row
 * is off by at most 2^-38 of the call's largest factor), and accumulates dx and dw
 * in fp32.
 * Every sum has a fixed order: the same call gives the same bits.
 *
 * What a call writes (loss and lse; dx and dw; its workspace) must not overlap
 * anything else that it takes; such calls are refused.  (Rows of one matrix may lie
 * between those of another at the same stride.)
 *
 * Streams, errors and the library workspace are as in gemm.h: calls are
 * asynchronous on args.stream (else the thread's gemm_set_stream; GEMM_NULL_STREAM:
 * HIP's null stream), return a
 * GEMM_* status, launch nothing on a negative one, and gemm_last_error() says
 * why.  They enqueue kernels only and can be captured; with workspace = NULL the
 * library workspace must have been sized by an eager call before.
 */
#ifndef DGW_GEMM_LOSS_H
#define DGW_GEMM_LOSS_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_LOSS_XENT    0u
#define GEMM_LOSS_DISTILL 1u

/* type of the teacher's logits */
#define GEMM_LOSS_FP32 0u
#define GEMM_LOSS_BF16 1u
#define GEMM_LOSS_FP16 2u

/* type of dw */
#define GEMM_LOSS_DW_SAME       0u   /* the operands' type, overwritten          */
#define GEMM_LOSS_DW_FP32       1u   /* fp32, overwritten                        */
#define GEMM_LOSS_DW_FP32_ADD   2u   /* fp32, added to what is there             */

#define GEMM_LOSS_MAX_T       (1 << 24)
#define GEMM_LOSS_MAX_V       (1 << 21)
#define GEMM_LOSS_MAX_H       (1 << 20)
#define GEMM_LOSS_MAX_TV      ((int64_t)1 << 37)   /* T * V: the tiles of one launch */
#define GEMM_LOSS_MAX_TH      ((int64_t)1 << 37)   /* T * H                           */
#define GEMM_LOSS_MAX_ENTRIES 1024

/*
 * Arguments; zero-initialise, then fill what the call needs.
 *   x, w:      device, 16-byte aligned rows; ldx, ldw: elements between rows (0:
 *              packed; else at least the row's length, a multiple of 8, at most 2^21).
 *   T, V, H:   T >= 0, V >= 1, H a multiple of 8 >= 8; V a multiple of 8 for GEMM_B_KN;
 *              at most GEMM_LOSS_MAX_*.
 *   layout:    GEMM_B_NK or GEMM_B_KN, combined with GEMM_BF16 or GEMM_FP16.
 *   kind:      GEMM_LOSS_XENT or GEMM_LOSS_DISTILL.
 *   target:    device int64 [T] (XENT).     ignore_index: the target of rows to leave out.
 *   z_loss:    zeta >= 0 (XENT).
 *   entries:   K, 1 .. GEMM_LOSS_MAX_ENTRIES (DISTILL).
 *   teacher_index:  device int64 [T,K], packed (DISTILL).
 *   teacher_logits: device [T,K], packed, of teacher_type (DISTILL).
 *   temperature:    tau > 0 (DISTILL); tau^2 must be a finite fp32 above 0 too.
 *   loss:      device fp32 [T], written by gemm_loss_forward.
 *   lse:       device fp32 [T], written by gemm_loss_forward, read by gemm_loss_backward.
 *   grad:      device fp32 [T], the gradient g of each row's loss (backward).
 *   dx:        device [T,H] of the operands' type, lddx as ldx; NULL: not computed.
 *   dw:        device, w's layout, of dw_type, lddw as ldw (fp32: a multiple of 4); NULL: not computed.
 *   stream, workspace, workspace_bytes: as in gemm_args_t, except that the
 *              workspace need not be cleared; gemm_loss_plan_t.workspace_bytes is needed.
 *   num_cus:   plan for this many compute units, at most 65536 (0: the device's).
 */
typedef struct gemm_loss_args_t {
    const void *x;
    const void *w;
    int64_t T, V, H;
    int64_t ldx, ldw;
    uint32_t layout;
    uint32_t kind;
    const int64_t *target;
    int64_t ignore_index;
    float z_loss;
    int32_t entries;
    const int64_t *teacher_index;
    const void *teacher_logits;
    uint32_t teacher_type;
    float temperature;
    float *loss;
    float *lse;
    const float *grad;
    void *dx;
    int64_t lddx;
    void *dw;
    int64_t lddw;
    uint32_t dw_type;
    int32_t num_cus;
    void *stream;
    void *workspace;
    size_t workspace_bytes;
} gemm_loss_args_t;

/* How a call runs (host arithmetic only). */
typedef struct gemm_loss_plan_t {
    int32_t tile_v, tile_t;         /* logits tile: vocabulary entries x rows             */
    int32_t num_cus;
    int32_t pieces;                 /* backward: pieces of the vocabulary                  */
    int64_t piece;                  /* backward: vocabulary entries per piece (the last: the rest) */
    int32_t dx_tile_h, dx_tile_t;   /* backward: tile of dx                                */
    int32_t dx_splits;              /* backward: slices of a piece's entries summed apart  */
    int32_t dw_tile_p, dw_tile_q;   /* backward: tile of dw (columns x rows as stored)     */
    int32_t dw_splits;              /* backward: slices of the rows summed apart           */
    int64_t workspace_bytes;
} gemm_loss_plan_t;

/* gemm_loss_plan -- plan the forward (backward = 0) or backward (1) call of `args`
 * for num_cus compute units (1 .. 65536).  Reads sizes, layout, kind, entries, dx, dw and
 * dw_type only (the pointers for being NULL or not). */
int gemm_loss_plan(const gemm_loss_args_t *args, int32_t backward, int32_t num_cus, gemm_loss_plan_t *out);

/* gemm_loss_forward -- loss and lse.  T == 0: nothing to do. */
int gemm_loss_forward(const gemm_loss_args_t *args);

/* gemm_loss_backward -- dx and dw from grad and the forward pass's lse.  T == 0:
 * dw is zero-filled (GEMM_LOSS_DW_FP32_ADD: left as it is). */
int gemm_loss_backward(const gemm_loss_args_t *args);

#ifdef __cplusplus
}
#endif

#endif /* DGW_GEMM_LOSS_H */
