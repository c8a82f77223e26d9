// ffn.h -- launch interface of the gated feed-forward kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_ffn.h"
#include "loss.h"

namespace dgw {

// Tiles are named as the losses' (P x Q).  Of the forward kernel's P rows one half are
// gate features, the other the same features of up.
struct FfnGate {
    int T, F, H;
    LossMatrix gate, up, x;     // gate and up: F rows; x: k contiguous
    uint32_t act;
    uint16_t *h;                // [T][ldh], the product of the activation and up
    int64_t ldh, part;          // tiles of at most LOSS_FEW rows write what the rounding left out `part` elements on
    uint16_t *kept_gate, *kept_up;   // nullptr: not kept
    int64_t ld_gate, ld_up;
};
hipError_t launch_ffn_gate(int dtype, int tile, const FfnGate &p, hipStream_t stream);

// The whole forward call of at most FFN_VEC_T rows and weights with k contiguous: h [T][F]
// is a workspace, fp32; p's own h is not used.
constexpr int FFN_VEC_T = 4;
hipError_t launch_ffn_vec(int dtype, const FfnGate &p, const LossMatrix &down, float *h, uint16_t *y, int64_t ldy, hipStream_t stream);

// dh = dy . w_down, turned into dg, du and h where it stands.
struct FfnSlope {
    int T, F, H;
    LossMatrix down, dy;        // down: F rows; dy: k contiguous
    uint32_t act;
    const uint16_t *gate, *up;
    int64_t ld_gate, ld_up;
    uint16_t *dg, *du, *h;      // [T][ld]
    int64_t ld, part;           // as ldh and part above
};
hipError_t launch_ffn_slope(int dtype, int tile, const FfnSlope &p, hipStream_t stream);

// out[q][p] = sum_f gate[p][f] dg[q][f] + up[p][f] du[q][f] in the operands' type, or
// (splits > 1) the slices' slots as launch_loss_product writes them.  gate and up have
// one ld, dg and du too.
struct FfnSum {
    LossMatrix gate, up, dg, du;
    int F, splits;
    void *out;
    int64_t ldo;
};
hipError_t launch_ffn_sum(int dtype, int tile, const FfnSum &p, hipStream_t stream);

// out[q][p] = sum over T rows of P[t][p] Q[t][q], for up to three weights in one launch,
// and one that joins where the rows are cut into `splits` slices (by way of `slots`,
// loss_slots_bytes() for each weight, one behind the other); out_kind LO_16, LO_F32 or
// LO_F32_ADD.
struct FfnWeights {
    struct One {
        LossMatrix P, Q;   // rows contiguous
        void *out;         // nullptr: left out
        int64_t ldo;
    } one[3];
    int T, out_kind, splits;
    float *slots;   // nullptr: splits is 1
};
hipError_t launch_ffn_weights(int dtype, int tile, const FfnWeights &p, hipStream_t stream);

}  // namespace dgw
