// lora.h -- launch interface of the adapters' kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_lora.h"
#include "loss.h"

namespace dgw {

// Each row's adapter: adapter[row] in 0 .. count - 1, none (negative) or out of range.
struct LoraRows {
    const int64_t *adapter;
    int T;
    int count;
    const float *scale;   // per adapter, or nullptr: 1
};

// One low-rank side of every adapter: element (r, k) as in LossMatrix, the next
// adapter `stride` elements on.
struct LoraFactor {
    LossMatrix first;   // R rows
    int64_t stride;
};

// partial[s][row][r] = sum over slice s of k of x[row][k] f[r][k] with the row's own
// adapter's f, [splits][T][R] fp32, unscaled; rows without an adapter are left as they
// are.  `lists` workgroups of a group of rows share its adapters.
struct LoraLow {
    LoraRows rows;
    LoraFactor f;
    LossMatrix x;       // T rows, k contiguous
    int R, K;
    int lists, splits;
    float *partial;     // launch_lora_lows: nullptr leaves this product out
    bool by_rows;       // launch_lora_few, launch_lora_lows: a workgroup for a row and eight ranks, splits is 1
};
enum LoraLowTile : int { LL_32x64 = 0, LL_64x64, LL_128x64 };   // R x rows; 32: k contiguous only
int lora_low_tile(int R, bool kc);
int lora_low_rows(int tile);    // R rows of a tile
hipError_t launch_lora_low(int dtype, const LoraLow &p, hipStream_t stream);
// Both products of a backward call, one with a factor stored k contiguous and one not,
// and, masks != nullptr, masks[a][slab]: which of rows 64 slab .. + 63 have adapter a.
hipError_t launch_lora_lows(int dtype, const LoraLow &s, const LoraLow &ds, uint64_t *masks, hipStream_t stream);

// The slices' sums, scaled, as the type holds them, [T][R]; a null low is not kept.
struct LoraLowJoin {
    LoraRows rows{};
    int R = 0;
    const float *s = nullptr, *ds = nullptr;
    int s_splits = 1, ds_splits = 1;
    uint16_t *s_low = nullptr, *ds_low = nullptr;
};
hipError_t launch_lora_low_join(int dtype, const LoraLowJoin &p, hipStream_t stream);

// out[q][p] = sum_k P[p][k] x[q][k] + sum_r f[p][r] low[q][r], f the row's adapter's and low its
// scaled partial sums as the type holds them.  The first `whole` tiles are written whole in
// the operands' type; the rest in `splits` slices to `slots`, which launch_lora_join or
// launch_lora_outers adds up.  Rows whose adapter is out of range are NaN.
struct LoraProduct {
    LoraRows rows;
    LossMatrix P, x;
    LoraFactor f;       // P.rows rows, stored as P is
    const float *partial;   // nullptr: without the adapters' part, which the join of few rows adds (whole is 0)
    int low_splits;
    int K, R, splits, whole;
    float *slots;       // nullptr: splits is 1
    void *out;
    int64_t ldo;
};
enum LoraTile : int { LP_128x128 = LT_128x128, LP_256x256 = LT_256x256, LP_64x64 = LT_64x64, LP_64x128 = LT_64x128, LP_64x32 = 100 };
LossTileShape lora_tile_shape(int tile);
// `join` runs beside the tiles.
hipError_t launch_lora_product(int dtype, int tile, const LoraProduct &p, const LoraLowJoin &join, hipStream_t stream);
hipError_t launch_lora_join(int dtype, int tile, const LoraProduct &p, hipStream_t stream);

// Few rows (at most LORA_FEW_T rows, ranks of at most LORA_FEW_R): out and the narrow
// product that it needs in two launches, every tile through `slots` (whole is 0); f's part
// is summed in fp32 from unrounded narrow rows.
constexpr int LORA_FEW_T = 256, LORA_FEW_R = 256;
hipError_t launch_lora_few(int dtype, int tile, const LoraProduct &p, const LoraLow &low, hipStream_t stream);
// The second of them, after launch_lora_product without partial.
hipError_t launch_lora_few_join(int dtype, int tile, const LoraProduct &p, const LoraLow &low, hipStream_t stream);

// out_a[q][p] = sum over the rows t of adapter a of P[t][p] Q[t][q], for every adapter.
// One of P and Q is the narrow side (R wide, `narrow_p` says which).
struct LoraOuter {
    LossMatrix P, Q;    // rows contiguous
    bool narrow_p;
    int T, count;
    const uint64_t *masks;
    int splits;
    float *partial;     // splits > 1: [splits][count][Q.rows][P.rows]
    int out_kind;       // LO_16, LO_F32, LO_F32_ADD
    void *out;          // [count][Q.rows][P.rows], rows ldo apart, adapters `stride`; nullptr: left out
    int64_t ldo, stride;
};
// da and db in one launch, one of them with a narrow P, and the join of a product's tail
// (of tiles `tile`) unless that is nullptr; with `few`, that of few rows.
hipError_t launch_lora_outers(int dtype, const LoraOuter &da, const LoraOuter &db, int tile, const LoraProduct *tail, const LoraLow *few,
                              hipStream_t stream);

}  // namespace dgw
