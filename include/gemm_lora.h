/*
 * gemm_lora.h -- a projection shared by many requests, each row of which may add a
 * low-rank adapter of its own, and its gradients (gfx950).
 *
 *   x [T,H] bf16/fp16; of the same type
 *   GEMM_B_NK:  w [N,H]   a [L,R,H]   b [L,N,R]
 *   GEMM_B_KN:  w [H,N]   a [L,H,R]   b [L,R,N]        (each matrix transposed)
 *   adapter [T] int64: row t's adapter a_t; negative: none      scale [L] fp32 or NULL (1)
 *
 * Forward (as written for GEMM_B_NK), c = scale[a_t]:
 *   s_t = c x_t . a[a_t]^T        y_t = x_t . w^T + s_t . b[a_t]^T
 * Backward, from dy [T,N]:
 *   ds_t = c dy_t . b[a_t]        dx_t = dy_t . w + ds_t . a[a_t]
 *   da[l] = sum_{t: a_t = l} ds_t (x) x_t        db[l] = sum_{t: a_t = l} dy_t (x) s_t
 * (w is shared and has no gradient here; gemm_ex computes one.)
 *
 * Rows may name adapters in any order; requests whose rows lie together cost least,
 * as a product tile goes over every adapter that occurs among its rows.  An adapter
 * that no row names is not read, and its da and db are zero.  A row whose adapter is
 * >= L has y and dx of NaN and no part in da and db: nothing is read out of range.
 * What x and dy hold in one row, infinities and NaN too, never reaches another row or
 * another adapter's da and db, and what an adapter holds reaches the rows that name it
 * and no others.  (A call with such an adapter beyond 128 rows takes two to four times
 * as long, with many of them up to ten times.)
 *
 * Arithmetic: products in fp32.  s and ds, the operands of the next products, are
 * rounded to the type once, after the scale, as tensors of the type would be (up to 256
 * rows y and dx may be made from them unrounded); y, dx,
 * and da and db of the type once each; y's and dx's two parts are one fp32 sum.
 * fp16 values beyond its range become infinities, as everywhere.
 * Every sum has a fixed order: the same call gives the same bits.
 *
 * What a call writes (y; dx, da and db; its workspace) must not overlap anything else
 * that it takes; such calls are refused.  (Rows of one matrix may lie between those of
 * another at the same stride.)
 *
 * Streams, errors and the library workspace are as in gemm.h: calls are
 * asynchronous on args.stream (else the thread's gemm_set_stream; GEMM_NULL_STREAM:
 * HIP's null stream), return a GEMM_* status, launch nothing on a negative one, and
 * gemm_last_error() says why.  They enqueue kernels only and can be captured; with
 * workspace = NULL the library workspace must have been sized by an eager call before.
 */
#ifndef DGW_GEMM_LORA_H
#define DGW_GEMM_LORA_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* type of da and db */
#define GEMM_LORA_DAB_SAME     0u   /* the operands' type, overwritten */
#define GEMM_LORA_DAB_FP32     1u   /* fp32, overwritten               */
#define GEMM_LORA_DAB_FP32_ADD 2u   /* fp32, added to what is there    */

#define GEMM_LORA_MAX_T        (1 << 24)
#define GEMM_LORA_MAX_H        (1 << 20)   /* H and N */
#define GEMM_LORA_MAX_R        1024
#define GEMM_LORA_MAX_ADAPTERS (1 << 16)
#define GEMM_LORA_MAX_TH       ((int64_t)1 << 37)   /* T * H, T * N and H * N      */
#define GEMM_LORA_MAX_LT       ((int64_t)1 << 34)   /* L * T (backward)            */
#define GEMM_LORA_MAX_LRH      ((int64_t)1 << 38)   /* L * R * H and L * R * N     */
#define GEMM_LORA_MAX_TR       ((int64_t)1 << 31)   /* T * R                       */
#define GEMM_LORA_MAX_TILES    ((int64_t)1 << 23)   /* backward: L ceil(R / 64) (ceil(H / 128) if da + ceil(N / 128) if db) */
#define GEMM_LORA_MAX_STRIDE   ((int64_t)1 << 40)   /* stride_a, stride_b          */

/*
 * Arguments; zero-initialise, then fill what the call needs.
 *   x, w:      device, 16-byte aligned rows; ldx, ldw: elements between rows (0:
 *              packed; else at least the row's length, a multiple of 8, at most 2^21).
 *   a, b:      device, 16-byte aligned, each adapter's matrix packed; stride_a,
 *              stride_b: elements between adapters (0: packed; else at least a matrix,
 *              a multiple of 8, at most GEMM_LORA_MAX_STRIDE).
 *   T, H, N, R, adapters: T >= 0; H, N and R multiples of 8 >= 8; adapters (L) >= 1; at
 *              most GEMM_LORA_MAX_*.
 *   layout:    GEMM_B_NK or GEMM_B_KN, combined with GEMM_BF16 or GEMM_FP16.
 *   adapter:   device int64 [T].        scale: device fp32 [L], NULL: 1.
 *   y:         device [T,N] of the operands' type, written by the forward call.
 *   dy:        device [T,N], read by the backward call.
 *   dx:        device [T,H]; NULL: not computed.
 *   da, db:    device, shaped as a and b, packed, of dab_type; each NULL: not computed.
 *   stream, workspace, workspace_bytes: as in gemm_args_t, except that the workspace
 *              need not be cleared; gemm_lora_plan_t.workspace_bytes is needed.
 *   num_cus:   plan for this many compute units, at most 65536 (0: the device's).
 */
typedef struct gemm_lora_args_t {
    const void *x;
    const void *w;
    const void *a;
    const void *b;
    const int64_t *adapter;
    const float *scale;
    int64_t T, H, N;
    int32_t R, adapters;
    int64_t ldx, ldw, stride_a, stride_b;
    uint32_t layout;
    uint32_t dab_type;
    void *y;
    int64_t ldy;
    const void *dy;
    int64_t lddy;
    void *dx;
    int64_t lddx;
    void *da;
    void *db;
    int32_t num_cus;
    void *stream;
    void *workspace;
    size_t workspace_bytes;
} gemm_lora_args_t;

/* How a call runs (host arithmetic only). */
typedef struct gemm_lora_plan_t {
    int32_t num_cus;
    int32_t low_tile_r, low_splits, low_lists;   /* s (backward: ds): rank x 64 rows (8: a row by itself); slices of k; workgroups over a tile's adapters */
    int32_t out_tile_p, out_tile_t;              /* tile of y (backward: dx)                  */
    int32_t out_splits;                          /* slices of k of the tiles behind the first out_whole */
    int32_t dab_splits;                          /* backward: slices of the rows for da and db */
    int64_t out_whole;                           /* tiles computed whole                      */
    int64_t workspace_bytes;
} gemm_lora_plan_t;

/* gemm_lora_plan -- plan the forward (backward = 0) or backward (1) call of `args` for
 * num_cus compute units (1 .. 65536).  Reads sizes, layout, dx, da, db and dab_type only
 * (the pointers for being NULL or not). */
int gemm_lora_plan(const gemm_lora_args_t *args, int32_t backward, int32_t num_cus, gemm_lora_plan_t *out);

/* gemm_lora_forward -- y.  T == 0: nothing to do. */
int gemm_lora_forward(const gemm_lora_args_t *args);

/* gemm_lora_backward -- dx, da and db.  T == 0: da and db are zero-filled
 * (GEMM_LORA_DAB_FP32_ADD: left as they are). */
int gemm_lora_backward(const gemm_lora_args_t *args);

#ifdef __cplusplus
}
#endif

#endif /* DGW_GEMM_LORA_H */
