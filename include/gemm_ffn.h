/*
 * gemm_ffn.h -- the gated feed-forward block and its gradients (gfx950).
 *
 *   x [T,H] bf16/fp16, and three weights of the same type:
 *   GEMM_B_NK:  w_gate, w_up [F,H]   w_down [H,F]
 *   GEMM_B_KN:  w_gate, w_up [H,F]   w_down [F,H]        (each transposed)
 *
 * Forward (as written for GEMM_B_NK):
 *   g = x . w_gate^T   u = x . w_up^T   h = act(g) u   y = h . w_down^T
 * Both first products, the activation and the product h run in one kernel; g and
 * u reach memory only where the caller asks for them (gate and up, which the
 * backward call reads).
 * Backward, from dy and the kept gate and up:
 *   dh = dy . w_down   dg = dh u act'(g)   du = dh act(g)   h = act(g) u
 *   dx = dg . w_gate + du . w_up
 *   dw_gate = dg^T . x   dw_up = du^T . x   dw_down = dy^T . h   (stored as the weights are)
 * with dg, du and h made by one kernel from dy . w_down where it stands.
 *
 * act:  GEMM_FFN_SILU  g / (1 + exp(-g))      GEMM_FFN_GELU  g Phi(g), Phi the standard
 *       normal CDF (erf to 1.5e-7)            GEMM_FFN_RELU  max(g, 0), slope 0 at 0
 *
 * Arithmetic: products, activations and their slopes in fp32.  h, dg and du, the
 * operands of the next products, are rounded to the type once (up to 64 rows: to the
 * sum of two such values, as nothing averages there and the weights' streams are
 * the time; the forward call of up to 4 rows with GEMM_B_NK keeps h in fp32); kept gate and up, y, dx and weight gradients of the type once each.
 * fp16 values beyond its range become infinities, as everywhere.
 * Every sum has a fixed order: the same call gives the same bits.
 *
 * What a call writes (y, gate and up; dx and the weights' gradients; its workspace)
 * must not overlap anything else that it takes; such calls are refused.  (Rows of one
 * matrix may lie between those of another at the same stride.)
 *
 * Streams, errors and the library workspace are as in gemm.h: calls are
 * asynchronous on args.stream (else the thread's gemm_set_stream; GEMM_NULL_STREAM:
 * HIP's null stream), return a GEMM_* status, launch nothing on a negative one, and
 * gemm_last_error() says why.  They enqueue kernels only and can be captured; with
 * workspace = NULL the library workspace must have been sized by an eager call before.
 */
#ifndef DGW_GEMM_FFN_H
#define DGW_GEMM_FFN_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GEMM_FFN_SILU 0u
#define GEMM_FFN_GELU 1u
#define GEMM_FFN_RELU 2u

/* type of the weights' gradients */
#define GEMM_FFN_DW_SAME     0u   /* the operands' type, overwritten */
#define GEMM_FFN_DW_FP32     1u   /* fp32, overwritten               */
#define GEMM_FFN_DW_FP32_ADD 2u   /* fp32, added to what is there    */

#define GEMM_FFN_MAX_T  (1 << 24)
#define GEMM_FFN_MAX_H  (1 << 20)
#define GEMM_FFN_MAX_F  (1 << 20)
#define GEMM_FFN_MAX_TH ((int64_t)1 << 37)   /* T * H, T * F and H * F: the tiles of one launch */

/*
 * Arguments; zero-initialise, then fill what the call needs.
 *   x, w_*:    device, 16-byte aligned rows; ld*: elements between rows (0: packed;
 *              else at least the row's length, a multiple of 8, at most 2^21).
 *   T, H, F:   T >= 0, H and F multiples of 8 >= 8; at most GEMM_FFN_MAX_*.
 *   layout:    GEMM_B_NK or GEMM_B_KN, combined with GEMM_BF16 or GEMM_FP16.
 *   act:       GEMM_FFN_SILU, GEMM_FFN_GELU or GEMM_FFN_RELU.
 *   gate, up:  device [T,F] of the operands' type; written by the forward call (both or
 *              neither: NULL), read by the backward call.
 *   y:         device [T,H], written by the forward call.
 *   dy:        device [T,H], read by the backward call.
 *   dx:        device [T,H]; NULL: not computed.
 *   dw_*:      device, stored as the weight is, of dw_type (fp32: ld a multiple of 4);
 *              each NULL: not computed.
 *   stream, workspace, workspace_bytes: as in gemm_args_t, except that the workspace
 *              need not be cleared; gemm_ffn_plan_t.workspace_bytes is needed.
 *   num_cus:   plan for this many compute units, at most 65536 (0: the device's).
 */
typedef struct gemm_ffn_args_t {
    const void *x;
    const void *w_gate;
    const void *w_up;
    const void *w_down;
    int64_t T, H, F;
    int64_t ldx, ldw_gate, ldw_up, ldw_down;
    uint32_t layout;
    uint32_t act;
    void *gate;
    void *up;
    int64_t ldgate, ldup;
    void *y;
    int64_t ldy;
    const void *dy;
    int64_t lddy;
    void *dx;
    int64_t lddx;
    void *dw_gate;
    void *dw_up;
    void *dw_down;
    int64_t lddw_gate, lddw_up, lddw_down;
    uint32_t dw_type;
    int32_t num_cus;
    void *stream;
    void *workspace;
    size_t workspace_bytes;
} gemm_ffn_args_t;

/* How a call runs (host arithmetic only). */
typedef struct gemm_ffn_plan_t {
    int32_t num_cus;
    int32_t parts;                       /* 16-bit parts of h, dg and du (0: h in fp32)      */
    int32_t first_tile_f, first_tile_t;  /* features x rows of the kernel that makes h (backward: dg, du and h) */
    int32_t out_tile_h, out_tile_t;      /* tile of y (backward: dx)                         */
    int32_t out_splits;                  /* slices of F summed apart                         */
    int32_t dw_tile_p, dw_tile_q;        /* backward: tile of the weights' gradients (columns x rows as stored) */
    int32_t dw_splits;                   /* backward: slices of the rows summed apart        */
    int64_t workspace_bytes;
} gemm_ffn_plan_t;

/* gemm_ffn_plan -- plan the forward (backward = 0) or backward (1) call of `args` for
 * num_cus compute units (1 .. 65536).  Reads sizes, layout, act, dx, dw_*, dw_type,
 * ldw_gate and ldw_up only (the pointers for being NULL or not). */
int gemm_ffn_plan(const gemm_ffn_args_t *args, int32_t backward, int32_t num_cus, gemm_ffn_plan_t *out);

/* gemm_ffn_forward -- y (and gate and up).  T == 0: nothing to do. */
int gemm_ffn_forward(const gemm_ffn_args_t *args);

/* gemm_ffn_backward -- dx and the weights' gradients.  T == 0: the gradients are
 * zero-filled (GEMM_FFN_DW_FP32_ADD: left as they are). */
int gemm_ffn_backward(const gemm_ffn_args_t *args);

#ifdef __cplusplus
}
#endif

#endif /* DGW_GEMM_FFN_H */
