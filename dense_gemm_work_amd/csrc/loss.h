// loss.h -- launch interface of the vocabulary-loss kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_loss.h"

namespace dgw {

// Tile shapes (P x Q; P: the dimension contiguous in the result).  The tiles of
// few rows take a Q operand with k contiguous, the 32- and 64-row ones a P
// operand with k contiguous too.
enum LossTile : int { LT_128x128 = 0, LT_256x256, LT_32x32, LT_128x32, LT_64x64, LT_64x128, LT_128x64 };
struct LossTileShape {
    int p, q, per_cu;   // rows of P and Q, workgroups resident per CU
};
LossTileShape loss_tile_shape(int tile);

// An operand as it lies in memory: element (row, k) at base[row * ld + k]
// (kc) or base[k * ld + row].
struct LossMatrix {
    const uint16_t *base;
    int64_t ld;
    int rows;
    bool kc;
    int64_t part = 0;   // elements from the first 16-bit part to the second (0: one part)
};

// Up to this many rows dz is the sum of two 16-bit parts.
constexpr int LOSS_FEW = 64;

// The rows' sparse targets as the logits' epilogues read them.  XENT: the int64
// target itself, weight 1.  DISTILL: a row's entries {index, probability} sorted
// by bucket of the vocabulary (64 buckets of `width` entries), and where each
// bucket starts among them.
constexpr int LOSS_BUCKETS = 64;
constexpr int LOSS_STARTS = LOSS_BUCKETS + 2;   // per row: 64 starts, the end, and one to keep rows aligned
struct LossTargets {
    const int64_t *target;
    const uint2 *entries;     // [T][stride]
    const uint16_t *starts;   // [T][LOSS_STARTS]
    int stride;
    int width;
};

// Forward statistics of a logits launch: per tile of the vocabulary and row, the
// maximum logit, the sum of exp2((z - max) c) and the targets' weighted logits.
struct LossStats {
    float *max, *sum, *dot;   // [tiles_v][T]
};

// What the rows' contributions to the logits' gradient follow from.
struct LossRows {
    int64_t V;
    float zeta, tau, inv_tau;
    const int64_t *target;   // XENT
    int64_t ignore;
    const float *entropy;    // DISTILL
    const float *grad, *lse;
};

struct LossProblem {
    int T, V, H;
    float c;              // log2(e) / tau
    LossMatrix x, w;      // w offset to the piece's first entry
    int64_t v0;           // that entry's index
    LossTargets targets;
};

// Logits of p.T rows over p.V entries, reduced to statistics.
hipError_t launch_loss_stats(int dtype, int tile, const LossProblem &p, const LossStats &s, hipStream_t stream);

// Logits again, as their gradient dz [T][ldd] (16 bits; ldd a multiple of 8,
// zeros behind p.V), times *scale when scale != nullptr.  The tiles of at most
// LOSS_FEW rows write what the rounding left out, rounded too, `part` elements on.
hipError_t launch_loss_dz(int dtype, int tile, const LossProblem &p, const LossRows &rows, const float *scale, uint16_t *dz,
                          int64_t ldd, int64_t part, hipStream_t stream);

// out[q][p] = sum_k P[p][k] Q[q][k], times *unscale when unscale != nullptr.
enum LossOut : int {
    LO_16 = 0,         // the operands' type
    LO_F32 = 1,        // fp32
    LO_F32_ADD = 2,    // fp32, added to out
    LO_SLOTS = 3,      // fp32 partials per (slice, tile), register order
    LO_SLOTS_ADD = 4,  // the same, added to what the slots hold
};
struct LossProduct {
    LossMatrix P, Q;
    int K;
    int splits;
    int out_kind;
    void *out;
    int64_t ldo;
    const float *unscale;   // not applied to slots
};
// The tiles of at most LOSS_FEW rows take a Q of two parts, the others one of one.
hipError_t launch_loss_product(int dtype, int tile, const LossProduct &p, hipStream_t stream);

// The same for K <= LOSS_FEW (one slab), both operands' rows contiguous and one of
// them of two parts, on at most about `workgroups` persistent workgroups (the splits
// and slots do not apply).
hipError_t launch_loss_outer(int dtype, const LossProduct &p, int workgroups, hipStream_t stream);

// out from the slots of `splits` slices: out_kind LO_16, LO_F32 or LO_F32_ADD.
hipError_t launch_loss_join(int dtype, int tile, const LossProduct &p, const float *slots, hipStream_t stream);
int64_t loss_slots_bytes(int tile, int64_t rows_p, int64_t rows_q, int splits);

// The teacher's entries as LossTargets holds them, and sum q log q per row (NaN
// where an entry is out of range; -infinity marks rows without entries).
hipError_t launch_loss_teacher(int64_t T, int K, int64_t V, const int64_t *index, const void *logits, uint32_t type,
                               float tau, uint2 *entries, uint16_t *starts, float *entropy, hipStream_t stream);
int loss_bucket_width(int64_t V);

// loss and lse from the statistics of `tiles` tiles.
hipError_t launch_loss_finish(const gemm_loss_args_t &a, int tiles, const LossStats &s, const float *entropy,
                              hipStream_t stream);

// scale[0], the power of two multiplied into an fp16 dz, and scale[1] = 1 / scale[0].
hipError_t launch_loss_scale(const LossRows &rows, int64_t T, float *scale, hipStream_t stream);

hipError_t launch_loss_zero(void *out, int64_t rows, int64_t row_bytes, int64_t ld_bytes, hipStream_t stream);

}  // namespace dgw
