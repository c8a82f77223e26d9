// loss_kernels.hip -- gfx950 kernels of the vocabulary losses (gemm_loss.h).
//
// Forward: loss_stats computes a tile of logits (vocabulary x rows) with the loop
// of tile.h and reduces it where it stands: per row the maximum, the sum of
// exponentials and the targets' weighted logits, 12 bytes per row and tile
// instead of the tile itself.  loss_finish joins the tiles' statistics.
// Backward, per piece of the vocabulary: loss_dz computes the logits again and
// writes their gradient in 16 bits, loss_product multiplies it with w (dx) and x
// (dw).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "loss.h"
#include "tile.h"

namespace dgw {

using namespace tile;

namespace {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float INF = __builtin_inff();

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

struct LogitParams {
    Matrix w, x;
    int T, V, H;
    int64_t v0;
    float c;
    Grid g;
    LossTargets targets;
};

// Where a lane's row has its targets: the int64 target, or the range of its
// entries whose buckets meet the wave's part of the tile.
struct TargetRange {
    int64_t target;
    const uint2 *entries;
    int at, end;
};

// `first`: the vocabulary index of the wave's first row of P.
template <int WAVE_P>
__device__ __forceinline__ TargetRange target_range(const LossTargets &t, int64_t first, int64_t row, bool valid) {
    TargetRange r{-1, nullptr, 0, 0};
    if (!valid) return r;
    if (t.target) {
        r.target = t.target[row];
        return r;
    }
    const uint16_t *s = t.starts + row * LOSS_STARTS;
    const int lo = (int)first / t.width, hi = ((int)first + WAVE_P - 1) / t.width;
    r.entries = t.entries + row * t.stride;
    r.at = s[min(lo, LOSS_BUCKETS)];
    r.end = s[min(hi, LOSS_BUCKETS - 1) + 1];
    return r;
}

// A lane's registers of one block column, laid down in LDS so that they can be
// indexed: quad i of the lane at [i][lane], so every access is free of bank
// conflicts and no lane touches another's.  (Picking one of 64 registers by
// comparisons costs 128 instructions an entry; with 128 entries a row dz of
// 1024 x 32768 x 1536 took 177 us that way.)
template <class L>
struct LaneArray {
    f32x4 *quads;
    static constexpr int BYTES = L::RB * 1024;   // per wave
    __device__ __forceinline__ LaneArray(char *lds, const L &loop)
        : quads(reinterpret_cast<f32x4 *>(lds + loop.wave * BYTES) + loop.lane) {
        static_assert(L::NW * BYTES <= L::LDS_BYTES, "an array for every wave");
    }
    __device__ __forceinline__ void put(const typename L::Acc &acc, int j) {
#pragma unroll
        for (int i = 0; i < L::RB; ++i) quads[i * 64] = acc.v[i][j];
    }
    __device__ __forceinline__ void get(typename L::Acc &acc, int j) const {
#pragma unroll
        for (int i = 0; i < L::RB; ++i) acc.v[i][j] = quads[i * 64];
    }
    __device__ __forceinline__ float &at(int slot) { return reinterpret_cast<float *>(quads + (slot >> 2) * 64)[slot & 3]; }
};

// Whether any lane of the wave may have a target in the wave's part of the tile.
template <int WAVE_P>
__device__ __forceinline__ bool any_target(const LossTargets &t, const TargetRange &r, int64_t first) {
    return __any(t.target ? r.target >= first && r.target < first + WAVE_P : r.at < r.end);
}

// Calls f(slot, weight) in the lanes that hold a target's logit, for the row's
// targets in the wave's part of the tile, in their order: slot 4 i + e is
// register e of block i.  Of the four lanes that share a row each calls f for the
// entries it holds.  Entries are read four at a time, so their loads overlap.
template <int WAVE_P, class F>
__device__ __forceinline__ void for_targets(const LossTargets &t, const TargetRange &r, int64_t first, int group, F &&f) {
    auto visit = [&](int64_t at, float weight) {
        if (at < 0 || at >= WAVE_P || (((int)at >> 2) & 3) != group || weight == 0.0f) return;
        const int p = (int)at;
        f((p >> 4) * 4 + (p & 3), weight);
    };
    if (t.target) {
        if (r.target >= 0) visit(r.target - first, 1.0f);
        return;
    }
    for (int k = r.at; k < r.end; k += 4) {
        uint2 e[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) e[x] = r.entries[min(k + x, r.end - 1)];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (k + x < r.end) visit((int64_t)(int)e[x].x - first, __uint_as_float(e[x].y));
    }
}

// ---------------------------------------------------------------------------
// Forward statistics of one tile.  A lane holds 4 RB logits of one row per block
// column, so maximum and sum run over registers; the four lanes that share a row
// meet by two lane exchanges, the WP waves through LDS.
// ---------------------------------------------------------------------------
template <class L>
__global__ __launch_bounds__(L::NT, 2) void loss_stats(LogitParams p, LossStats s) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    static_assert(3 * L::WP * L::TQ * 4 <= L::LDS_BYTES, "the waves' statistics fit");
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    loop.run_any(p.w, p0, p.x, q0, p.H, 0, p.g.slabs, acc);
    if (p0 + L::TP > p.V) {   // entries beyond the vocabulary take no part
#pragma unroll
        for (int i = 0; i < L::RB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p0 + loop.p_of(i, e) >= p.V)
#pragma unroll
                    for (int j = 0; j < L::CB; ++j) acc.v[i][j][e] = -INF;
    }
    float *st = reinterpret_cast<float *>(lds);
    const int group = loop.lane >> 4;
    const int64_t first = p.v0 + p0 + loop.wp * L::WAVE_P;
    TargetRange range[L::CB];
#pragma unroll
    for (int j = 0; j < L::CB; ++j) range[j] = target_range<L::WAVE_P>(p.targets, first, q0 + loop.q_of(j), q0 + loop.q_of(j) < p.T);
    float max[L::CB], sum[L::CB], dot[L::CB];
    LaneArray<L> array(lds, loop);
    if (loop.active())
#pragma unroll
        for (int j = 0; j < L::CB; ++j) {
            float m = -INF;
#pragma unroll
            for (int i = 0; i < L::RB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) m = fmaxf(m, acc.v[i][j][e]);
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            // the maximum is subtracted first, exactly: its own exponential is then 1, the
            // sum at least 1 and no loss negative.  (z c - round(m c) would keep the
            // rounding of m c, 1e-5 at logits of 250.)
            const float top = m == -INF ? 0.0f : m;   // a row of -infinity sums to 0
            float se = 0.0f;
#pragma unroll
            for (int i = 0; i < L::RB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) se += exp2_fast((acc.v[i][j][e] - top) * p.c);
            float d = 0.0f;
            if (any_target<L::WAVE_P>(p.targets, range[j], first)) {
                array.put(acc, j);
                for_targets<L::WAVE_P>(p.targets, range[j], first, group,
                                       [&](int slot, float weight) { d = __builtin_fmaf(weight, array.at(slot), d); });
            }
            max[j] = m;
            se += __shfl_xor(se, 16);
            sum[j] = se + __shfl_xor(se, 32);
            d += __shfl_xor(d, 16);
            dot[j] = d + __shfl_xor(d, 32);
        }
    __syncthreads();   // the lanes' arrays give way to the statistics
    if (loop.active() && group == 0)
#pragma unroll
        for (int j = 0; j < L::CB; ++j) {
            const int at = loop.wp * L::TQ + loop.q_of(j);
            st[at] = max[j];
            st[L::WP * L::TQ + at] = sum[j];
            st[2 * L::WP * L::TQ + at] = dot[j];
        }
    __syncthreads();
    for (int t = threadIdx.x; t < L::TQ; t += L::NT) {
        if (q0 + t >= p.T) break;
        float m = st[t];
#pragma unroll
        for (int w = 1; w < L::WP; ++w) m = fmaxf(m, st[w * L::TQ + t]);
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int w = 0; w < L::WP; ++w) {
            const float mw = st[w * L::TQ + t], sw = st[(L::WP + w) * L::TQ + t];
            sum += mw == -INF ? sw : sw * exp2_fast((mw - m) * p.c);
            dot += st[(2 * L::WP + w) * L::TQ + t];
        }
        const int64_t at = (int64_t)tp * p.T + q0 + t;
        s.max[at] = m;
        s.sum[at] = sum;
        s.dot[at] = dot;
    }
}

// ---------------------------------------------------------------------------
// 16-bit stores of a tile: packed into LDS row by row (16-byte chunk c of row r
// at c ^ r), then whole rows go out 16 bytes a lane.  NT: non-temporal, for results
// that the call does not read again (dw of 64 x 50001 x 2048: 62 against 52 us).
// ---------------------------------------------------------------------------
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == 0) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, f16x2));
}

// v less its rounding to the type.
template <int DT>
__device__ __forceinline__ float remainder16(float v) {
    if constexpr (DT == 0) return v - (float)(__bf16)v;
    else return v - (float)(_Float16)v;
}

// The LDS must be free.  Chunks at or beyond cols8 (a multiple of 8) and rows at
// or beyond rows_q are not stored.
template <int DT, bool NT, class L>
__device__ __forceinline__ void store16(const L &loop, const typename L::Acc &acc, char *lds, uint16_t *out, int64_t ld,
                                        int64_t p0, int64_t q0, int64_t cols8, int64_t rows_q, float u = 1.0f) {
    constexpr int CH = L::TP / 8;   // chunks per row
    static_assert(L::TP * L::TQ * 2 <= L::LDS_BYTES, "the tile fits");
    if (loop.active())
#pragma unroll
    for (int j = 0; j < L::CB; ++j) {
        const int r = loop.q_of(j);
#pragma unroll
        for (int i = 0; i < L::RB; ++i)
        {
            const int p = loop.p_of(i, 0);
            const int chunk = (p >> 3) ^ (r & (CH - 1));
            *reinterpret_cast<u32x2 *>(lds + r * (2 * L::TP) + chunk * 16 + (p & 4) * 2) =
                u32x2{pack2<DT>(acc.v[i][j][0] * u, acc.v[i][j][1] * u), pack2<DT>(acc.v[i][j][2] * u, acc.v[i][j][3] * u)};
        }
    }
    __syncthreads();
#pragma unroll 4
    for (int f = threadIdx.x; f < L::TQ * CH; f += L::NT) {
        const int r = f / CH, c = f % CH;
        if (q0 + r < rows_q && p0 + 8 * c < cols8) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(lds + r * (2 * L::TP) + ((c ^ (r & (CH - 1))) << 4));
            u32x4 *at = reinterpret_cast<u32x4 *>(out + (q0 + r) * ld + p0 + 8 * c);
            if constexpr (NT) __builtin_nontemporal_store(v, at);
            else *at = v;
        }
    }
}

// ---------------------------------------------------------------------------
// What a row contributes to the logits' gradient, dz = a p - b q (0 when !on).
// ---------------------------------------------------------------------------
struct RowFactors {
    float lse;
    float a, b;
    bool on;
};
__device__ __forceinline__ RowFactors row_factors(const LossRows &p, int64_t row) {
    const float lse = p.lse[row], g = p.grad[row];
    RowFactors r{lse, 0.0f, 0.0f, true};
    if (p.target) {
        const int64_t y = p.target[row];
        const float bad = y < 0 || y >= p.V ? __builtin_nanf("") : 0.0f;
        r.on = y != p.ignore;
        r.a = g * __builtin_fmaf(2.0f * p.zeta, lse, 1.0f) + bad;
        r.b = g;
    } else {
        const float h = p.entropy[row];
        r.on = h != -INF;
        r.a = h != h ? h : g * p.tau;
        r.b = g * p.tau;
    }
    if (!r.on) r.lse = r.a = r.b = 0.0f;
    return r;
}

// ---------------------------------------------------------------------------
// The logits' gradient of one tile: dz = a p - b q, p = exp(z / tau - lse).  lse is
// subtracted before the factor log2 e: at a sure row's target z / tau = lse, p = 1 and
// dz = 0.  (z c - round(lse log2 e) left up to 1e-5 there at logits of 250.)
// dz is rounded to the operands' type, the matrix instructions' input: with many rows
// dx and dw are then off by 0.0024 (bf16) or 0.0003 (fp16) of their size, rounded
// themselves 0.0017 or 0.0002; a second part would cost each of their products
// twice.  A row's gradient is mostly its target's entry, so with few rows nothing
// averages (0.0042 at two rows), and there the streams of w and dw are the time: the
// tiles of at most LOSS_FEW rows write the remainder too.
// ---------------------------------------------------------------------------
template <int DT, class L>
__global__ __launch_bounds__(L::NT, 2) void loss_dz(LogitParams p, LossRows rows, const float *scale, uint16_t *dz,
                                                 int64_t ldd, int64_t part) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    loop.run_any(p.w, p0, p.x, q0, p.H, 0, p.g.slabs, acc);
    const float S = scale ? scale[0] : 1.0f, inv_tau = rows.inv_tau;
    const int64_t first = p.v0 + p0 + loop.wp * L::WAVE_P;
    TargetRange range[L::CB];
#pragma unroll
    for (int j = 0; j < L::CB; ++j) range[j] = target_range<L::WAVE_P>(p.targets, first, q0 + loop.q_of(j), q0 + loop.q_of(j) < p.T);
    LaneArray<L> array(lds, loop);
    if (loop.active())
#pragma unroll
    for (int j = 0; j < L::CB; ++j) {
        const int64_t row = q0 + loop.q_of(j);
        const RowFactors r = row_factors(rows, row < p.T ? row : p.T - 1);
        const float a = r.a * S, b = r.b * S;
#pragma unroll
        for (int i = 0; i < L::RB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc.v[i][j][e] = a * exp2_fast(__builtin_fmaf(acc.v[i][j][e], inv_tau, -r.lse) * LOG2E);
        if (any_target<L::WAVE_P>(p.targets, range[j], first)) {
            array.put(acc, j);
            for_targets<L::WAVE_P>(p.targets, range[j], first, loop.lane >> 4,
                                   [&](int slot, float weight) { array.at(slot) -= b * weight; });
            array.get(acc, j);
        }
        // rows without a target, whatever their logits are, and the padding
        // behind the vocabulary
        const bool ragged = p0 + L::TP > p.V;
        if (ragged || __any(!r.on)) {
#pragma unroll
            for (int i = 0; i < L::RB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!r.on || p0 + loop.p_of(i, e) >= p.V) acc.v[i][j][e] = 0.0f;
        }
    }
    __syncthreads();   // the lanes' arrays give way to the packed tile
    store16<DT, false>(loop, acc, lds, dz, ldd, p0, q0, ldd, p.T);
    if constexpr (L::TQ <= LOSS_FEW) {
#pragma unroll
        for (int i = 0; i < L::RB; ++i)
#pragma unroll
            for (int j = 0; j < L::CB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.v[i][j][e] = remainder16<DT>(acc.v[i][j][e]);
        __syncthreads();
        store16<DT, false>(loop, acc, lds, dz + part, ldd, p0, q0, ldd, p.T);
    }
}

// ---------------------------------------------------------------------------
// Plain products: dx and dw.
// ---------------------------------------------------------------------------
struct ProductParams {
    Matrix P, Q;
    int K;
    Grid g;
    int out_kind;
    void *out;
    int64_t ldo;
    const float *unscale;
};

// Slot of (slice, tile): a wave's blocks one after the other, each 64 float4 (one
// a lane), so every access moves 1 KiB of contiguous memory.
template <class L>
__device__ __forceinline__ f32x4 *slot_base(float *slots, const Grid &g, int tp, int tq, int split, int wave, int lane) {
    const int64_t tile = ((int64_t)split * g.tiles_q + tq) * g.tiles_p + tp;
    return reinterpret_cast<f32x4 *>(slots + tile * (L::TP * L::TQ)) + wave * (L::RB * L::CB * 64) + lane;
}

template <int DT, class L>
__global__ __launch_bounds__(L::NT, L::WAVES) void loss_product(ProductParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    const int s0 = (int)((int64_t)p.g.slabs * split / p.g.splits), s1 = (int)((int64_t)p.g.slabs * (split + 1) / p.g.splits);
    loop.run_any(p.P, p0, p.Q, q0, p.K, s0, s1, acc);
    if (p.out_kind >= LO_SLOTS) {
        if (!loop.active()) return;
        f32x4 *slot = slot_base<L>(static_cast<float *>(p.out), p.g, tp, tq, split, loop.wave, loop.lane);
        const bool add = p.out_kind == LO_SLOTS_ADD;
#pragma unroll
        for (int i = 0; i < L::RB; ++i) {
#pragma unroll
            for (int j = 0; j < L::CB; ++j) {
                f32x4 *at = slot + (i * L::CB + j) * 64;
                *at = add ? acc.v[i][j] + *at : acc.v[i][j];
            }
            __builtin_amdgcn_sched_barrier(0);   // one block row's loads in flight: no more registers are free
        }
        return;
    }
    const float u = p.unscale ? *p.unscale : 1.0f;
    if (p.out_kind == LO_16) {
        store16<DT, true>(loop, acc, lds, static_cast<uint16_t *>(p.out), p.ldo, p0, q0, (p.P.rows + 7) & ~7, p.Q.rows, u);
        return;
    }
    float *out = static_cast<float *>(p.out);
    if (!loop.active()) return;
    const bool add = p.out_kind == LO_F32_ADD;
#pragma unroll
    for (int i = 0; i < L::RB; ++i) {
#pragma unroll
        for (int j = 0; j < L::CB; ++j) {
            const int64_t col = p0 + loop.p_of(i, 0), row = q0 + loop.q_of(j);
            if (row < p.Q.rows && col < p.P.rows) {
                f32x4 *at = reinterpret_cast<f32x4 *>(out + row * p.ldo + col);
                *at = add ? acc.v[i][j] * u + *at : acc.v[i][j] * u;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// ---------------------------------------------------------------------------
// dw of at most 64 rows: one slab of k, so the stores are the cost.  A workgroup
// keeps its 128 rows of P in registers and walks over tiles of Q: the next tile's
// slab is on its way while this one is multiplied, and a tile's stores while the
// next is.  64 x 50001 x 2048, dz in one part: 49 us with a workgroup per tile (each
// waits out its slab's latency alone), 39 us this way (5.3 TB/s written); in two
// parts 47.5 us (4.3 TB/s), in fp32 107 us, added to fp32 180 us (4.5 TB/s read and
// written).  64 x 32000 x 2048, w [H,V]: 26.9 us (4.9 TB/s).
// One operand is dz in two parts.  As P both lie in registers; as Q they take two of
// three places in LDS, so that two workgroups still fit a CU: the next tile's first
// part goes into the third while this tile is multiplied, its second part into the
// place that this tile's first part leaves.
// ---------------------------------------------------------------------------
template <int DT, int KIND, bool PARTS_P>
__global__ __launch_bounds__(256, 2) void loss_outer(ProductParams p) {
    using Op = Operand<false, 128, 4>;
    constexpr int PP = PARTS_P ? 2 : 1, PQ = 3 - PP;                    // parts of P and Q
    constexpr int OUT = 128 * 128 * 2, CH = 16;                         // packed result tile in bytes; chunks a row
    constexpr int STORES = KIND == LO_16 ? 8 : 16;                      // per thread
    __shared__ __attribute__((aligned(16))) char lds[OUT + (PQ + 1) * Op::SLAB];
    static_assert(PP * Op::SLAB <= OUT, "P's slabs borrow the result's place");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wp = wave & 1, wq = wave >> 1;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
    // the grid is a multiple of tiles_p: a workgroup stays with its tile of P
    const int tp = (int)blockIdx.x % p.g.tiles_p, step = (int)gridDim.x / p.g.tiles_p;
    int tq = (int)blockIdx.x / p.g.tiles_p;
    const int64_t p0 = (int64_t)tp * 128;
    auto load = [&](const Matrix &m, int part, int64_t row0, uint32_t dst) {
        Op o;
        o.init(m, row0, p.K, wave, lane);
        const i32x4 r = o.rsrc(0, part * 2 * m.part);
#pragma unroll
        for (int x = 0; x < Op::LOADS; ++x) o.template load<false>(r, 0, x, dst + wave * Op::LOADS * 1024);
    };
    uint32_t place[PQ], spare = lds0 + OUT + PQ * Op::SLAB;             // of this tile's parts of Q; free
#pragma unroll
    for (int x = 0; x < PP; ++x) load(p.P, x, p0, lds0 + x * Op::SLAB);
#pragma unroll
    for (int x = 0; x < PQ; ++x) load(p.Q, x, (int64_t)tq * 128, place[x] = lds0 + OUT + x * Op::SLAB);
    wait_vm_lgkm<0>();
    barrier();
    u32x4 pf[PP][2][4];
#pragma unroll
    for (int x = 0; x < PP; ++x)
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pf[x][st][i] = Op::fragment(Op::address(lds0, wp * 64, lane, i) + x * Op::SLAB + Op::constant(0, st));
    uint32_t qa[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) qa[j] = Op::address(0, wq * 64, lane, j);
    wait_vm_lgkm<0>();   // P's fragments are in registers before its place is written
    const float u = p.unscale ? *p.unscale : 1.0f;
    const int cols = (int)min((int64_t)128, ((p.P.rows + 7) & ~7) - p0);
    bool first = true;
    for (; tq < p.g.tiles_q; tq += step) {
        const int64_t q0 = (int64_t)tq * 128;
        const bool more = tq + step < p.g.tiles_q;
        // This tile's slabs are older than the last tile's stores, every one of which
        // is issued whether it is inside the result or not.  After the barrier the
        // spare place and the result's are free.
        __builtin_amdgcn_sched_barrier(0);
        if (first) wait_vm_lgkm<0>();
        else wait_vm_lgkm<STORES>();
        first = false;
        barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (more) load(p.Q, 0, q0 + (int64_t)step * 128, spare);
        f32x4 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int y = PQ - 1; y >= 0; --y) {
                u32x4 qf[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) qf[j] = Op::fragment(place[y] + qa[j] + Op::constant(0, st));
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = PP - 1; x >= 0; --x) acc[i][j] = mfma<DT>(pf[x][st][i], qf[j], acc[i][j]);
            }
        if constexpr (KIND == LO_16) {
            // the packed tile, 16-byte chunk c of row r at c ^ r
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = wq * 64 + j * 16 + (lane & 15);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = wp * 64 + i * 16 + 4 * (lane >> 4);
                    *reinterpret_cast<u32x2 *>(lds + r * 256 + (((c >> 3) ^ (r & (CH - 1))) << 4) + (c & 4) * 2) =
                        u32x2{pack2<DT>(acc[i][j][0] * u, acc[i][j][1] * u), pack2<DT>(acc[i][j][2] * u, acc[i][j][3] * u)};
                }
            }
        }
        if constexpr (KIND == LO_16 || PQ == 2) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt((15 | (3 << 14)) | (7 << 4));   // this wave's LDS operations; its loads go on
            barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (PQ == 2) {
            if (more) load(p.Q, 1, q0 + (int64_t)step * 128, place[0]);
            __builtin_amdgcn_sched_barrier(0);
        }
        const int rows = (int)min((int64_t)128, p.Q.rows - q0);
        if constexpr (KIND == LO_16) {
            const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
                static_cast<uint16_t *>(p.out) + q0 * p.ldo + p0, (short)0, (int)(((rows - 1) * p.ldo + cols) * 2), (int)RSRC_DW3);
#pragma unroll
            for (int x = 0; x < STORES; ++x) {
                const int f = threadIdx.x + 256 * x, r = f / CH, c = f % CH;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(lds + r * 256 + ((c ^ (r & (CH - 1))) << 4));
                const uint32_t off = r < rows && 8 * c < cols ? (uint32_t)(r * p.ldo + 8 * c) * 2 : OOB;
                __builtin_amdgcn_raw_buffer_store_b128(v, out, (int)off, 0, 2);   // non-temporal
            }
        } else {   // four consecutive floats a lane; fp32 written through the caches (117 against 139 us for 64 x 32000 x 2048)
            const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
                static_cast<float *>(p.out) + q0 * p.ldo + p0, (short)0, (int)(((rows - 1) * p.ldo + cols) * 4), (int)RSRC_DW3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = wq * 64 + j * 16 + (lane & 15);
                uint32_t off[4];
                u32x4 old[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = wp * 64 + i * 16 + 4 * (lane >> 4);
                    off[i] = r < rows && c < cols ? (uint32_t)(r * p.ldo + c) * 4 : OOB;
                    if constexpr (KIND == LO_F32_ADD) old[i] = __builtin_amdgcn_raw_buffer_load_b128(out, (int)off[i], 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 v = acc[i][j] * u;
                    if constexpr (KIND == LO_F32_ADD) v += __builtin_bit_cast(f32x4, old[i]);
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), out, (int)off[i], 0, 0);
                }
            }
        }
        const uint32_t left = place[PQ - 1];   // the next tile's parts: in the spare place, and in the first one's
        if constexpr (PQ == 2) place[1] = place[0];
        place[0] = spare;
        spare = left;
    }
}

// The slices' slots added in slice order.  One thread per float4 of a slot.
template <int DT, class L>
__global__ __launch_bounds__(256) void loss_join(ProductParams p, const float *slots) {
    constexpr int QUADS = L::TP * L::TQ / 4;
    const int64_t id = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (id >= (int64_t)p.g.tiles_p * p.g.tiles_q * QUADS) return;
    const int tile = (int)(id / QUADS), f = (int)(id % QUADS);
    const int tp = tile % p.g.tiles_p, tq = tile / p.g.tiles_p;
    const int lane = f & 63, block = (f >> 6) % (L::RB * L::CB), wave = (f >> 6) / (L::RB * L::CB);
    const int i = block / L::CB, j = block % L::CB, wp = wave % L::WP, wq = wave / L::WP;
    const int64_t col = (int64_t)tp * L::TP + wp * L::WAVE_P + i * 16 + 4 * (lane >> 4);
    const int64_t row = (int64_t)tq * L::TQ + wq * L::WAVE_Q + j * 16 + (lane & 15);
    if (row >= p.Q.rows || col >= p.P.rows) return;
    const int64_t step = (int64_t)p.g.tiles_p * p.g.tiles_q * QUADS;
    const f32x4 *at = reinterpret_cast<const f32x4 *>(slots) + id;
    f32x4 v = at[0];
    int s = 1;
    for (; s + 4 <= p.g.splits; s += 4) {   // four loads in flight, added in order
        const f32x4 a = at[s * step], b = at[(s + 1) * step], c = at[(s + 2) * step], d = at[(s + 3) * step];
        v = (((v + a) + b) + c) + d;
    }
    for (; s < p.g.splits; ++s) v += at[s * step];
    v *= p.unscale ? *p.unscale : 1.0f;
    if (p.out_kind == LO_16) {
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + row * p.ldo + col) =
            u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        return;
    }
    f32x4 *out = reinterpret_cast<f32x4 *>(static_cast<float *>(p.out) + row * p.ldo + col);
    if (p.out_kind == LO_F32_ADD) v += *out;
    *out = v;
}

// ---------------------------------------------------------------------------
// Small kernels around the products.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

struct TeacherParams {
    int64_t T, V;
    int K, width;
    const int64_t *index;
    const void *logits;
    uint32_t type;
    float inv_tau;
    uint2 *entries;
    uint16_t *starts;
    float *entropy;
};

__device__ __forceinline__ float teacher_logit(const TeacherParams &p, int64_t at) {
    if (p.type == GEMM_LOSS_FP32) return static_cast<const float *>(p.logits)[at];
    if (p.type == GEMM_LOSS_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p.logits)[at] << 16);
    return (float)static_cast<const _Float16 *>(p.logits)[at];
}

// One wave per row: the softmax over its entries, then a counting sort of them
// by bucket, entries of one bucket in the order they came.  The row's maximum is
// taken of the logits as they are and subtracted before the division by tau: a
// finite logit stays finite at any tau (the lowest value over 0.5 would not), and
// the largest entry's argument is 0.
__global__ __launch_bounds__(256) void loss_teacher(TeacherParams p) {
    __shared__ int counts[4][LOSS_BUCKETS];
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    int *count = counts[threadIdx.x >> 6];
    if (row >= p.T) return;
    const int64_t base = row * p.K;
    float m = -INF;
    bool bad = false;
    for (int k = lane; k < p.K; k += 64) {
        const int64_t i = p.index[base + k];
        if (i < 0) continue;
        const float t = teacher_logit(p, base + k);
        bad |= i >= p.V || t != t;
        m = fmaxf(m, t);
    }
    m = wave_max(m);
    bad = __any(bad);
    const bool none = m == -INF;
    float total = 0.0f, dot = 0.0f;   // sum e, sum e t
    for (int k = lane; k < p.K; k += 64) {
        if (none || p.index[base + k] < 0) continue;
        const float t = (teacher_logit(p, base + k) - m) * p.inv_tau;
        const float e = t == -INF ? 0.0f : expf(t);
        total += e;
        dot += e > 0.0f ? e * t : 0.0f;
    }
    total = wave_sum(total);
    dot = wave_sum(dot);
    // sum q log q = sum e t / total - log total
    if (lane == 0) p.entropy[row] = bad ? __builtin_nanf("") : none ? -INF : dot / total - logf(total);

    // each lane's bucket and its rank among the lanes of the same bucket (-1: no entry)
    auto place = [&](int k, int &bucket, int &rank, bool &last) {
        const int64_t i = k < p.K ? p.index[base + k] : -1;
        const bool on = i >= 0 && i < p.V && !none;
        bucket = on ? (int)i / p.width : -1;
        uint64_t same = __ballot(on);
#pragma unroll
        for (int b = 0; b < 6; ++b) {
            const uint64_t set = __ballot((bucket >> b) & 1);
            same &= (bucket >> b) & 1 ? set : ~set;
        }
        rank = on ? __popcll(same & ((1ull << lane) - 1)) : -1;
        last = on && (same >> lane) == 1;
    };
    // the wave's LDS operations run in program order; the fences keep the compiler to it
    count[lane] = 0;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    const int rounds = (p.K + 63) / 64;
    for (int c = 0; c < rounds; ++c) {
        int bucket, rank;
        bool last;
        place(c * 64 + lane, bucket, rank, last);
        if (last) count[bucket] += rank + 1;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    }
    const int mine = count[lane];
    int upto = mine;   // entries in buckets 0 .. lane
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(upto, o);
        if (lane >= o) upto += x;
    }
    p.starts[row * LOSS_STARTS + lane] = (uint16_t)(upto - mine);
    if (lane == 63) p.starts[row * LOSS_STARTS + 64] = (uint16_t)upto;
    count[lane] = upto - mine;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    for (int c = 0; c < rounds; ++c) {
        const int k = c * 64 + lane;
        int bucket, rank;
        bool last;
        place(k, bucket, rank, last);
        if (rank >= 0) {
            const int at = count[bucket] + rank;
            const float t = (teacher_logit(p, base + k) - m) * p.inv_tau;
            const float q = t == -INF ? 0.0f : expf(t) / total;
            p.entries[base + at] = uint2{(uint32_t)p.index[base + k], __float_as_uint(q)};
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (last) count[bucket] += rank + 1;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    }
}

struct FinishParams {
    int64_t T, V;
    int tiles;
    float c, inv_tau, tau2, zeta;
    LossStats s;
    const float *entropy;
    const int64_t *target;
    int64_t ignore;
    float *loss, *lse;
};

// Block of 256 threads: `per` rows (a power of two), 256 / per threads a row.
__global__ __launch_bounds__(256) void loss_finish(FinishParams p, int per) {
    __shared__ float sm[256], ss[256], sd[256];
    const int r = threadIdx.x & (per - 1), part = threadIdx.x / per, parts = 256 / per;
    const int64_t row = (int64_t)blockIdx.x * per + r;
    float m = -INF, sum = 0.0f, dot = 0.0f;
    // the sums of (m, sum) and (mi, si); a NaN sum stays one, a part whose maximum
    // is -infinity has sum 0
    auto join = [&](float mi, float si) {
        const float top = fmaxf(m, mi);
        sum = (m == -INF ? sum : sum * exp2_fast((m - top) * p.c)) + (mi == -INF ? si : si * exp2_fast((mi - top) * p.c));
        m = top;
    };
    if (row < p.T) {
        for (int i = part; i < p.tiles; i += parts) {
            const int64_t at = (int64_t)i * p.T + row;
            join(p.s.max[at], p.s.sum[at]);
            dot += p.s.dot[at];
        }
    }
    for (int half = parts / 2; half; half /= 2) {   // a tree over the row's threads
        sm[threadIdx.x] = m;
        ss[threadIdx.x] = sum;
        sd[threadIdx.x] = dot;
        __syncthreads();
        if (part < half) {
            const int o = threadIdx.x + half * per;
            join(sm[o], ss[o]);
            dot += sd[o];
        }
        __syncthreads();
    }
    if (part != 0 || row >= p.T) return;
    // loss from (max - target) + log(sum): exact where the target is the maximum
    const float log_sum = logf(sum);
    const float lse = m == -INF && sum == 0.0f ? -INF : __builtin_fmaf(m, p.inv_tau, log_sum);
    p.lse[row] = lse;
    float loss;
    if (p.target) {
        const int64_t y = p.target[row];
        loss = (m - dot) + log_sum;
        if (p.zeta != 0.0f) loss = __builtin_fmaf(p.zeta * lse, lse, loss);
        if (y < 0 || y >= p.V) loss = __builtin_nanf("");
        if (y == p.ignore) loss = 0.0f;
    } else {
        const float h = p.entropy[row];
        loss = h == -INF ? 0.0f : p.tau2 * (h + __builtin_fmaf(m - dot, p.inv_tau, log_sum));
    }
    p.loss[row] = loss;
}

// The fp16 scale: the power of two that brings the largest |a| or |b| into
// [2^13, 2^14), so dz, at most that in size, neither overflows nor loses the
// small probabilities to fp16's smallest values.  One block.
__global__ __launch_bounds__(1024) void loss_scale(LossRows p, int64_t T, float *scale) {
    __shared__ float part[16];
    float m = 0.0f;
    for (int64_t i = threadIdx.x; i < T; i += 1024) {
        const RowFactors r = row_factors(p, i);
        m = fmaxf(m, fmaxf(fabsf(r.a), fabsf(r.b)));
    }
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 1; i < 16; ++i) m = fmaxf(m, part[i]);
    int e = 0;
    if (m > 0.0f && m < INF) {
        e = 14 - (ilogbf(m) + 1);
        e = min(max(e, -120), 120);
    }
    scale[0] = ldexpf(1.0f, e);
    scale[1] = ldexpf(1.0f, -e);
}

__global__ __launch_bounds__(256) void loss_zero(char *out, int64_t rows, int64_t words, int64_t ld_bytes) {
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256)
            reinterpret_cast<uint32_t *>(out + r * ld_bytes)[i] = 0u;
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------
// 128 x 128: four waves of 64 x 64, two workgroups a CU.
// 256 x 256: eight waves of 128 x 64, one workgroup a CU.
// A third stage of P (all of the LDS then) lets P's loads, most of which miss the
// L2, travel for two iterations instead of one.  4096 x 131072 x 4096 on 256 x 256:
// logits 2.995 against 3.071 ms, dz and dx 6.22 against 6.48 ms; with both
// operands' rows contiguous (dw) 29 registers a lane spill instead of 16, dz and dw
// take 6.67 against 6.35 ms.  (Every 256 x 256 form spills some of its 256 registers:
// logits 6, of w [H,V] 11, dz and dx 2.)  On 128 x 128 tiles it pays for logits
// (333 x 50001 x 2048: 79.9 against 84.3 us; w [H,V]: 80.7 against 88.3) and for
// products of operands with k contiguous, not for the others (that shape's dz and
// dx: 168 against 164.5 us).
template <int TILE, int DT, bool PK, bool QK, bool LOGITS = false>
struct LoopOf;
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_128x128, DT, PK, QK, LOGITS> {
    using type = Loop<DT, PK, QK, 128, 128, 2, 2, QK && (PK || LOGITS) ? 3 : 2, 2>;
};
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_256x256, DT, PK, QK, LOGITS> {
    using type = Loop<DT, PK, QK, 256, 256, 2, 4, PK || QK ? 3 : 2, 2>;
};
// Few rows: ThinLoop tiles, several workgroups a CU for logits (48 to 80 KiB of LDS);
// dx, whose Q is dz in two parts, runs one a CU (96 KiB).
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_32x32, DT, PK, QK, LOGITS> {
    using type = ThinLoop<DT, PK, QK, 32, 32, 6>;
};
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_128x32, DT, PK, QK, LOGITS> {
    using type = ThinLoop<DT, PK, QK, 128, 32, 4, LOGITS ? 1 : 2>;
};
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_64x64, DT, PK, QK, LOGITS> {
    using type = ThinLoop<DT, PK, QK, 64, 64, 5>;
};
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_64x128, DT, PK, QK, LOGITS> {
    using type = ThinLoop<DT, PK, QK, 64, 128, 3>;
};
template <int DT, bool PK, bool QK, bool LOGITS>
struct LoopOf<LT_128x64, DT, PK, QK, LOGITS> {
    using type = ThinLoop<DT, PK, QK, 128, 64, 3, LOGITS ? 1 : 2>;
};
template <int DT>
using Loop128 = typename LoopOf<LT_128x128, DT, false, false>::type;
bool few_rows(int tile) { return loss_tile_shape(tile).q <= LOSS_FEW; }
template <class L_, int DT_>
struct Choice {
    using L = L_;
    static constexpr int DT = DT_;
};

Matrix matrix(const LossMatrix &m) { return Matrix{m.base, m.ld, m.rows, m.part}; }

template <class L>
Grid grid_of(int64_t rows_p, int64_t rows_q, int K, int splits) {
    Grid g;
    g.tiles_p = (int)((rows_p + L::TP - 1) / L::TP);
    g.tiles_q = (int)((rows_q + L::TQ - 1) / L::TQ);
    g.band = std::min(8, g.tiles_p);
    g.splits = splits;
    g.slabs = (K + KB - 1) / KB;
    return g;
}

unsigned blocks_of(const Grid &g) { return (unsigned)(g.tiles_p * g.tiles_q * g.splits); }

template <class L>
LogitParams logit_params(const LossProblem &p) {
    LogitParams q;
    q.w = matrix(p.w);
    q.x = matrix(p.x);
    q.T = p.T;
    q.V = p.V;
    q.H = p.H;
    q.v0 = p.v0;
    q.c = p.c;
    q.g = grid_of<L>(p.V, p.T, p.H, 1);
    q.targets = p.targets;
    return q;
}

template <class L>
hipError_t run_stats(const LossProblem &p, const LossStats &s, hipStream_t stream) {
    const LogitParams q = logit_params<L>(p);
    hipLaunchKernelGGL(loss_stats<L>, dim3(blocks_of(q.g)), dim3(L::NT), 0, stream, q, s);
    return hipGetLastError();
}
template <int DT, class L>
hipError_t run_dz(const LossProblem &p, const LossRows &rows, const float *scale, uint16_t *dz, int64_t ldd, int64_t part,
                  hipStream_t stream) {
    const LogitParams q = logit_params<L>(p);
    hipLaunchKernelGGL((loss_dz<DT, L>), dim3(blocks_of(q.g)), dim3(L::NT), 0, stream, q, rows, scale, dz, ldd, part);
    return hipGetLastError();
}
template <class L>
ProductParams product_params(const LossProduct &p) {
    return ProductParams{matrix(p.P), matrix(p.Q), p.K, grid_of<L>(p.P.rows, p.Q.rows, p.K, p.splits),
                         p.out_kind, p.out, p.ldo, p.unscale};
}
template <int DT, class L>
hipError_t run_product(const LossProduct &p, hipStream_t stream) {
    const ProductParams q = product_params<L>(p);
    hipLaunchKernelGGL((loss_product<DT, L>), dim3(blocks_of(q.g)), dim3(L::NT), 0, stream, q);
    return hipGetLastError();
}
template <int DT, class L>
hipError_t run_join(const LossProduct &p, const float *slots, hipStream_t stream) {
    const ProductParams q = product_params<L>(p);
    const int64_t quads = (int64_t)q.g.tiles_p * q.g.tiles_q * (L::TP * L::TQ / 4);
    const int64_t blocks = quads / 256, wide = std::min<int64_t>(blocks, 1 << 20);   // a dimension holds 2^32 threads
    hipLaunchKernelGGL((loss_join<DT, L>), dim3((unsigned)wide, (unsigned)((blocks + wide - 1) / wide)), dim3(256), 0, stream, q, slots);
    return hipGetLastError();
}

}  // namespace

LossTileShape loss_tile_shape(int tile) {
    switch (tile) {
    case LT_256x256: return {256, 256, 1};
    case LT_32x32: return {32, 32, 3};
    case LT_128x32: return {128, 32, 2};
    case LT_64x64: return {64, 64, 2};
    case LT_128x64: return {128, 64, 2};
    case LT_64x128: return {64, 128, 2};
    default: return {128, 128, 2};
    }
}

// f(loop type) for a tile, type and the operands' storage; an invalid value for
// what no call asks for.
template <int TILE, bool PK, bool QK, bool LOGITS, class F>
static hipError_t with_type(int dtype, F &&f) {
    return dtype == 0 ? f(Choice<typename LoopOf<TILE, 0, PK, QK, LOGITS>::type, 0>())
                      : f(Choice<typename LoopOf<TILE, 1, PK, QK, LOGITS>::type, 1>());
}
template <bool PK, bool QK, bool LOGITS = false, class F>
static hipError_t with_tile(int dtype, int tile, F &&f) {
    if constexpr (PK && QK && LOGITS) {   // their P slabs are too narrow for k-rows
        if (tile == LT_32x32) return with_type<LT_32x32, PK, QK, LOGITS>(dtype, f);
        if (tile == LT_64x64) return with_type<LT_64x64, PK, QK, LOGITS>(dtype, f);
        if (tile == LT_64x128) return with_type<LT_64x128, PK, QK, LOGITS>(dtype, f);
    }
    if constexpr (QK) {
        if (tile == LT_128x32) return with_type<LT_128x32, PK, QK, LOGITS>(dtype, f);
        if (tile == LT_128x64) return with_type<LT_128x64, PK, QK, LOGITS>(dtype, f);
    }
    switch (tile) {
    case LT_128x128: return with_type<LT_128x128, PK, QK, LOGITS>(dtype, f);
    case LT_256x256: return with_type<LT_256x256, PK, QK, LOGITS>(dtype, f);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_loss_stats(int dtype, int tile, const LossProblem &p, const LossStats &s, hipStream_t stream) {
    auto run = [&](auto c) { return run_stats<typename decltype(c)::L>(p, s, stream); };
    if (!p.x.kc) return hipErrorInvalidValue;
    return p.w.kc ? with_tile<true, true, true>(dtype, tile, run) : with_tile<false, true, true>(dtype, tile, run);
}

hipError_t launch_loss_dz(int dtype, int tile, const LossProblem &p, const LossRows &rows, const float *scale, uint16_t *dz,
                          int64_t ldd, int64_t part, hipStream_t stream) {
    auto run = [&](auto c) {
        using C = decltype(c);
        return run_dz<C::DT, typename C::L>(p, rows, scale, dz, ldd, part, stream);
    };
    if (!p.x.kc || few_rows(tile) != (part > 0)) return hipErrorInvalidValue;
    return p.w.kc ? with_tile<true, true, true>(dtype, tile, run) : with_tile<false, true, true>(dtype, tile, run);
}

hipError_t launch_loss_product(int dtype, int tile, const LossProduct &p, hipStream_t stream) {
    auto run = [&](auto c) {
        using C = decltype(c);
        return run_product<C::DT, typename C::L>(p, stream);
    };
    if (few_rows(tile) != (p.Q.part > 0) || p.P.part) return hipErrorInvalidValue;
    if (p.Q.kc) return p.P.kc ? with_tile<true, true>(dtype, tile, run) : with_tile<false, true>(dtype, tile, run);
    return p.P.kc ? hipErrorInvalidValue : with_tile<false, false>(dtype, tile, run);
}

template <int DT, bool PARTS_P>
static hipError_t run_outer(const ProductParams &q, int grid, hipStream_t stream) {
    if (q.out_kind == LO_16) hipLaunchKernelGGL((loss_outer<DT, LO_16, PARTS_P>), dim3(grid), dim3(256), 0, stream, q);
    else if (q.out_kind == LO_F32) hipLaunchKernelGGL((loss_outer<DT, LO_F32, PARTS_P>), dim3(grid), dim3(256), 0, stream, q);
    else hipLaunchKernelGGL((loss_outer<DT, LO_F32_ADD, PARTS_P>), dim3(grid), dim3(256), 0, stream, q);
    return hipGetLastError();
}

hipError_t launch_loss_outer(int dtype, const LossProduct &p, int workgroups, hipStream_t stream) {
    if (p.P.kc || p.Q.kc || p.K > LOSS_FEW || p.out_kind > LO_F32_ADD || (p.P.part > 0) == (p.Q.part > 0)) return hipErrorInvalidValue;
    static_assert(LOSS_FEW <= KB, "one slab of k");
    const ProductParams q = product_params<Loop128<0>>(p);
    const int grid = std::min(std::max(1, workgroups / q.g.tiles_p), q.g.tiles_q) * q.g.tiles_p;   // tiles_p < 2^14
    if (p.P.part) return dtype == 0 ? run_outer<0, true>(q, grid, stream) : run_outer<1, true>(q, grid, stream);
    return dtype == 0 ? run_outer<0, false>(q, grid, stream) : run_outer<1, false>(q, grid, stream);
}

hipError_t launch_loss_join(int dtype, int tile, const LossProduct &p, const float *slots, hipStream_t stream) {
    auto run = [&](auto c) {
        using C = decltype(c);
        return run_join<C::DT, typename C::L>(p, slots, stream);
    };
    return with_tile<true, true>(dtype, tile, run);   // the operands' storage does not matter here
}

int64_t loss_slots_bytes(int tile, int64_t rows_p, int64_t rows_q, int splits) {
    const LossTileShape s = loss_tile_shape(tile);
    return (rows_p + s.p - 1) / s.p * ((rows_q + s.q - 1) / s.q) * splits * (int64_t)s.p * s.q * 4;
}

int loss_bucket_width(int64_t V) { return (int)((V + LOSS_BUCKETS - 1) / LOSS_BUCKETS); }

hipError_t launch_loss_teacher(int64_t T, int K, int64_t V, const int64_t *index, const void *logits, uint32_t type,
                               float tau, uint2 *entries, uint16_t *starts, float *entropy, hipStream_t stream) {
    const TeacherParams p{T, V, K, loss_bucket_width(V), index, logits, type, 1.0f / tau, entries, starts, entropy};
    hipLaunchKernelGGL(loss_teacher, dim3((unsigned)((T + 3) / 4)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_loss_finish(const gemm_loss_args_t &a, int tiles, const LossStats &s, const float *entropy,
                              hipStream_t stream) {
    const float tau = a.kind == GEMM_LOSS_DISTILL ? a.temperature : 1.0f;
    FinishParams p{a.T, a.V, tiles, LOG2E / tau, 1.0f / tau, tau * tau, a.z_loss, s, entropy,
                   a.kind == GEMM_LOSS_XENT ? a.target : nullptr, a.ignore_index, a.loss, a.lse};
    // rows per block: 32 (whole cache lines) where that makes a block for every CU,
    // else fewer rows and more threads a row
    int per = 1;
    while (per < 32 && (int64_t)per * 256 < a.T) per *= 2;
    hipLaunchKernelGGL(loss_finish, dim3((unsigned)((a.T + per - 1) / per)), dim3(256), 0, stream, p, per);
    return hipGetLastError();
}

hipError_t launch_loss_scale(const LossRows &rows, int64_t T, float *scale, hipStream_t stream) {
    hipLaunchKernelGGL(loss_scale, dim3(1), dim3(1024), 0, stream, rows, T, scale);
    return hipGetLastError();
}

hipError_t launch_loss_zero(void *out, int64_t rows, int64_t row_bytes, int64_t ld_bytes, hipStream_t stream) {
    if (rows <= 0 || row_bytes <= 0) return hipSuccess;
    const int64_t words = row_bytes / 4;
    hipLaunchKernelGGL(loss_zero, dim3((unsigned)std::min<int64_t>((words + 255) / 256, 64), (unsigned)std::min<int64_t>(rows, 4096)),
                       dim3(256), 0, stream, static_cast<char *>(out), rows, words, ld_bytes);
    return hipGetLastError();
}

}  // namespace dgw
