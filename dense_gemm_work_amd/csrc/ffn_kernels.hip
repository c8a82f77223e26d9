// ffn_kernels.hip -- gfx950 kernels of the gated feed-forward block (gemm_ffn.h).
//
// Forward: ffn_gate computes a tile of x . w_gate^T and the same tile of
// x . w_up^T side by side (tile.h, PAIR), so a lane ends with both values of an
// element and writes act(g) u in 16 bits; g and u reach memory only where the
// caller keeps them.  Backward: ffn_slope computes a tile of dh = dy . w_down and
// turns it into dg = dh u act'(g), du = dh act(g) and h = act(g) u.  The products
// of h, dg and du with the weights and x are those of loss_kernels.hip.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "ffn.h"
#include "tile.h"
#include "tile_store.h"
#include "vec.h"

namespace dgw {

using namespace tile;

namespace {

constexpr float LOG2E = 1.44269504088896340736f;

// ---------------------------------------------------------------------------
// act(g) and act'(g) in fp32, branch free.
//   silu: g p, p = 1 / (1 + exp(-g));              p (1 + g (1 - p))
//   gelu: g Phi(g);                                Phi(g) + g phi(g)
//   relu: max(g, 0);                               [g > 0]
// Phi is (1 + erf(g / sqrt 2)) / 2 with erfc from the rational approximation of
// Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26 (absolute error
// 1.5e-7), the negative side from erfc itself, as the GEMM's epilogue does.
// ---------------------------------------------------------------------------
struct Act {
    float value, slope;
};
template <uint32_t ACT>
__device__ __forceinline__ Act activation(float g) {
    if constexpr (ACT == GEMM_FFN_SILU) {
        const float e = __builtin_amdgcn_exp2f(-g * LOG2E);
        const float p = __builtin_amdgcn_rcpf(1.0f + e);
        return {g * p, p * __builtin_fmaf(g, 1.0f - p, 1.0f)};
    } else if constexpr (ACT == GEMM_FFN_GELU) {
        const float x = fabsf(g) * 0.70710678118654752f, t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
        float poly = __builtin_fmaf(1.061405429f, t, -1.453152027f);
        poly = __builtin_fmaf(poly, t, 1.421413741f);
        poly = __builtin_fmaf(poly, t, -0.284496736f);
        poly = __builtin_fmaf(poly, t, 0.254829592f);
        const float bell = __builtin_amdgcn_exp2f(g * g * (-0.5f * LOG2E));   // exp(-g^2 / 2)
        const float q = 0.5f * poly * t * bell;
        const float phi = g >= 0.0f ? 1.0f - q : q;
        return {g * phi, __builtin_fmaf(g * bell, 0.39894228040143268f, phi)};
    } else {
        return {g <= 0.0f ? 0.0f : g, g <= 0.0f ? 0.0f : 1.0f};   // NaN stays
    }
}

// f(integral constant) for the activation: its branch is taken once, outside the loops.
template <class F>
__device__ __forceinline__ void with_act(uint32_t act, F &&f) {
    if (act == GEMM_FFN_SILU) f(std::integral_constant<uint32_t, GEMM_FFN_SILU>());
    else if (act == GEMM_FFN_GELU) f(std::integral_constant<uint32_t, GEMM_FFN_GELU>());
    else f(std::integral_constant<uint32_t, GEMM_FFN_RELU>());
}

// v in 16 bits at `to` and, TWO, what that left out, rounded too, `part` elements on
// (nothing where the first is infinite: infinity less infinity would make it NaN).
// The rest is taken from the stored bits: the compiler may fold the multiplication that
// made v into one of its conversions (v_fma_mixlo_f16) and not into another, and near a
// tie the two then round apart.
template <int DT, bool TWO>
__device__ __forceinline__ void store4(uint16_t *to, int64_t part, f32x4 v) {
    const u32x2 first = pack4<DT>(v);
    *reinterpret_cast<u32x2 *>(to) = first;
    if constexpr (TWO) {
        const f32x4 f = unpack4<DT>(first);
        f32x4 rest;
#pragma unroll
        for (int e = 0; e < 4; ++e) rest[e] = __builtin_isinf(f[e]) ? 0.0f : v[e] - f[e];
        *reinterpret_cast<u32x2 *>(to + part) = pack4<DT>(rest);
    }
}

struct GateParams {
    Matrix gate, up, x;
    int T, F, H;
    Grid g;
    uint32_t act;
    uint16_t *h, *kept_gate, *kept_up;
    int64_t ldh, part, ld_gate, ld_up;
};

// One matrix's half of a paired tile, as store16 takes a tile.
template <class L>
struct Half {
    static constexpr int TP = L::TP / 2, TQ = L::TQ, RB = L::RB / 2, CB = L::CB, NT = L::NT, LDS_BYTES = L::LDS_BYTES;
    struct Acc {
        f32x4 v[RB][CB];
    };
    const L &loop;
    __device__ __forceinline__ bool active() const { return loop.active(); }
    __device__ __forceinline__ int p_of(int i, int e) const { return loop.p_of(i, e); }
    __device__ __forceinline__ int q_of(int j) const { return loop.q_of(j); }
};

template <int DT, class L>
__global__ __launch_bounds__(L::NT, 2) void ffn_gate(GateParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * (L::TP / 2), q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    loop.run_any(loop.pick(p.gate, p.up), p0, p.x, q0, p.H, 0, p.g.slabs, acc);
    using V = Half<L>;
    const V half{loop};
    typename V::Acc out;
    auto take = [&](int kind) {
#pragma unroll
        for (int i = 0; i < V::RB; ++i)
#pragma unroll
            for (int j = 0; j < V::CB; ++j) out.v[i][j] = acc.v[2 * i + kind][j];
    };
    if (p.kept_gate) {
        take(0);
        store16<DT, true>(half, out, lds, p.kept_gate, p.ld_gate, p0, q0, p.F, p.T);
        __syncthreads();
        take(1);
        store16<DT, true>(half, out, lds, p.kept_up, p.ld_up, p0, q0, p.F, p.T);
        __syncthreads();
    }
    with_act(p.act, [&](auto A) {
#pragma unroll
        for (int i = 0; i < V::RB; ++i)
#pragma unroll
            for (int j = 0; j < V::CB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    out.v[i][j][e] = activation<decltype(A)::value>(acc.v[2 * i][j][e]).value * acc.v[2 * i + 1][j][e];
    });
    // h is rounded to the type here, once, as the operand of the next product's matrix
    // instructions: y is then off by sqrt 2 times its own rounding (0.0023 of its norm in bf16,
    // 0.0017 of them its own; 0.0003 in fp16).  A second part, as few rows have, would double
    // that product: 610 of 1740 us at 8192 x 4096 x 12288.
    store16<DT, false>(half, out, lds, p.h, p.ldh, p0, q0, p.F, p.T);
}

// Few rows: the halves' fp32 tiles meet in LDS ([row][TP + 4], 4 floats of padding
// against bank conflicts).  h is the sum of two 16-bit parts: with few rows the
// weights' stream is the time, and a second part costs it nothing.
template <int DT, class L>
__global__ __launch_bounds__(L::NT, L::WAVES) void ffn_gate_few(GateParams p) {
    constexpr int LD = L::TP + 4, QUADS = L::TP / 8;
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    static_assert(L::TQ * LD * 4 <= L::LDS_BYTES, "the tile fits");
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * (L::TP / 2), q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    loop.run_any(loop.pick(p.gate, p.up), p0, p.x, q0, p.H, 0, p.g.slabs, acc);
    float *tile = reinterpret_cast<float *>(lds);
    if (loop.active())
#pragma unroll
        for (int i = 0; i < L::RB; ++i)
#pragma unroll
            for (int j = 0; j < L::CB; ++j)
                *reinterpret_cast<f32x4 *>(tile + loop.q_of(j) * LD + loop.p_of(i, 0)) = acc.v[i][j];
    __syncthreads();
    with_act(p.act, [&](auto A) {
        for (int f = threadIdx.x; f < L::TQ * QUADS; f += L::NT) {
            const int64_t row = q0 + f / QUADS, col = p0 + 4 * (f % QUADS);
            if (row >= p.T || col >= p.F) continue;
            const float *at = tile + f / QUADS * LD + 4 * (f % QUADS);
            const f32x4 g = *reinterpret_cast<const f32x4 *>(at), u = *reinterpret_cast<const f32x4 *>(at + L::TP / 2);
            f32x4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = activation<decltype(A)::value>(g[e]).value * u[e];
            store4<DT, true>(p.h + row * p.ldh + col, p.part, h);
            if (p.kept_gate) {
                *reinterpret_cast<u32x2 *>(p.kept_gate + row * p.ld_gate + col) = pack4<DT>(g);
                *reinterpret_cast<u32x2 *>(p.kept_up + row * p.ld_up + col) = pack4<DT>(u);
            }
        }
    });
}

// At most VEC_T rows: four features a workgroup; h stays fp32.
template <int DT, int T>
__global__ __launch_bounds__(256) void ffn_gate_vec(GateParams p, float *h) {
    __shared__ float red[4][8][T];
    const int64_t f0 = (int64_t)blockIdx.x * 4;
    const uint16_t *w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = p.gate.base + (f0 + i) * p.gate.ld;
        w[4 + i] = p.up.base + (f0 + i) * p.up.ld;
    }
    dot_rows<DT>(w, Rows16<DT>{p.x.base, p.x.ld}, p.T, p.H, red);
    const int i = threadIdx.x & 3, t = threadIdx.x >> 2;
    if (t >= T || t >= p.T) return;
    const float g = joined(red, i, t), u = joined(red, 4 + i, t);
    with_act(p.act, [&](auto A) { h[(int64_t)t * p.F + f0 + i] = activation<decltype(A)::value>(g).value * u; });
    if (p.kept_gate) {
        p.kept_gate[t * p.ld_gate + f0 + i] = (uint16_t)pack2<DT>(g, 0.0f);
        p.kept_up[t * p.ld_up + f0 + i] = (uint16_t)pack2<DT>(u, 0.0f);
    }
}
template <int DT, int T>
__global__ __launch_bounds__(256) void ffn_down_vec(Matrix down, const float *h, int rows, int F, uint16_t *y, int64_t ldy) {
    __shared__ float red[4][4][T];
    const int64_t o0 = (int64_t)blockIdx.x * 4;
    const uint16_t *w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = down.base + (o0 + i) * down.ld;
    dot_rows<DT>(w, Rows32{h, F}, rows, F, red);
    const int i = threadIdx.x & 3, t = threadIdx.x >> 2;
    if (t < T && t < rows) y[t * ldy + o0 + i] = (uint16_t)pack2<DT>(joined(red, i, t), 0.0f);
}

struct SlopeParams {
    Matrix down, dy;
    int T, F, H;
    Grid g;
    uint32_t act;
    const uint16_t *gate, *up;
    int64_t ld_gate, ld_up;
    uint16_t *dg, *du, *h;
    int64_t ld, part;
};

// dg, du and h of one element.
struct Slopes {
    f32x4 dg, du, h;
};
template <int DT, uint32_t ACT>
__device__ __forceinline__ Slopes slopes(u32x2 gate, u32x2 up, f32x4 dh) {
    const f32x4 g = unpack4<DT>(gate), u = unpack4<DT>(up);
    Slopes s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const Act a = activation<ACT>(g[e]);
        s.dg[e] = dh[e] * u[e] * a.slope;
        s.du[e] = dh[e] * a.value;
        s.h[e] = u[e] * a.value;
    }
    return s;
}

// The epilogue of large tiles.  gate and up come, and dg, du and h go, as whole rows of a
// wave's part of the tile, 16 bytes a lane, by way of the wave's own share of the LDS
// (16-byte chunk c of row r at c ^ r); no wave waits for another.  16 rows at a time, the
// next 16 rows' gate and up on their way into the other of two buffers, dg and du over
// what they were made of.  The buffer's stores are issued whether a lane's row and
// chunk exist or not, so that the counts of what is in flight are known.  (8 bytes a
// lane straight from and to memory: 8192 x 4096 x 12288 997 us, 585 of them the product.)
// dg, du and h are rounded to the type once, as ffn_gate's h is and for its reason; second
// parts would double dx's and the weights' products, 3000 of 3690 us at that size.
template <int DT, uint32_t ACT, class L>
__device__ __forceinline__ void slope_rows(const SlopeParams &p, const L &loop, const typename L::Acc &acc, char *lds, int64_t p0, int64_t q0) {
    constexpr int ROW = 2 * L::WAVE_P, CH = ROW / 16, PART = 16 * ROW, N = PART / 1024;   // bytes a row and 16 rows; instructions
    constexpr int SHARE = 5 * PART;   // two buffers of gate and up, one of h
    static_assert(L::NW * SHARE <= L::LDS_BYTES && L::CB >= 2, "every wave's share fits");
    char *own = lds + loop.wave * SHARE;
    const uint32_t own0 = loop.lds0 + loop.wave * SHARE;
    const int lane = loop.lane;
    const int64_t pw = p0 + loop.wp * L::WAVE_P, qw = q0 + loop.wq * L::WAVE_Q;
    const int rows = (int)max((int64_t)0, min((int64_t)L::WAVE_Q, p.T - qw)), cols = (int)max((int64_t)0, min((int64_t)L::WAVE_P, p.F - pw));
    const bool any = rows > 0 && cols > 0;
    auto reach = [&](int64_t ld) { return any ? (uint32_t)(((rows - 1) * ld + cols) * 2) : 0u; };
    const i32x4 rg = make_rsrc(p.gate + (any ? qw * p.ld_gate + pw : 0), reach(p.ld_gate));
    const i32x4 ru = make_rsrc(p.up + (any ? qw * p.ld_up + pw : 0), reach(p.ld_up));
    // where lane's 16 bytes of instruction x lie: row of 16 and chunk
    auto row_of = [&](int x) { return (x * 1024 + lane * 16) / ROW; };
    auto chunk_of = [&](int x) { return ((x * 1024 + lane * 16) % ROW / 16) ^ (row_of(x) & (CH - 1)); };
    auto offset = [&](int j, int x, int64_t ld) {
        const int r = 16 * j + row_of(x), c = chunk_of(x);
        return r < rows && 8 * c < cols ? (uint32_t)(r * ld + 8 * c) * 2 : OOB;
    };
    auto fetch = [&](int j) {
        const uint32_t to = own0 + (j & 1) * 2 * PART;
#pragma unroll
        for (int x = 0; x < N; ++x) load_lds16(rg, to + x * 1024, offset(j, x, p.ld_gate));
#pragma unroll
        for (int x = 0; x < N; ++x) load_lds16(ru, to + PART + x * 1024, offset(j, x, p.ld_up));
    };
    auto send = [&](uint16_t *base, const char *from, int j) {
        const __amdgpu_buffer_rsrc_t out =
            __builtin_amdgcn_make_buffer_rsrc(base + (any ? qw * p.ld + pw : 0), (short)0, (int)reach(p.ld), (int)RSRC_DW3);
#pragma unroll
        for (int x = 0; x < N; ++x)
            __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4 *>(from + x * 1024 + lane * 16), out, (int)offset(j, x, p.ld), 0, 0);
    };
    fetch(0);
    fetch(1);
#pragma unroll
    for (int j = 0; j < L::CB; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        // behind this part's loads: the last one's stores and the next one's loads
        if (j == 0) wait_vm_lgkm<2 * N>();
        else if (j + 1 < L::CB) wait_vm_lgkm<5 * N>();
        else wait_vm_lgkm<3 * N>();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        char *g = own + (j & 1) * 2 * PART, *u = g + PART, *h = own + 4 * PART;
        const int r = lane & 15;
#pragma unroll
        for (int i = 0; i < L::RB; ++i) {
            const int c = 16 * i + 4 * (lane >> 4), at = r * ROW + (((c >> 3) ^ (r & (CH - 1))) << 4) + (c & 4) * 2;
            const Slopes s = slopes<DT, ACT>(*reinterpret_cast<const u32x2 *>(g + at), *reinterpret_cast<const u32x2 *>(u + at), acc.v[i][j]);
            *reinterpret_cast<u32x2 *>(g + at) = pack4<DT>(s.dg);
            *reinterpret_cast<u32x2 *>(u + at) = pack4<DT>(s.du);
            *reinterpret_cast<u32x2 *>(h + at) = pack4<DT>(s.h);
        }
        asm volatile("" ::: "memory");
        send(p.dg, g, j);
        send(p.du, u, j);
        send(p.h, h, j);
        __builtin_amdgcn_sched_barrier(0);
        if (j + 2 < L::CB) {
            __builtin_amdgcn_s_waitcnt((15 | (3 << 14)) | (7 << 4));   // this buffer has been read
            fetch(j + 2);
        }
    }
}

// Few rows: a lane's four consecutive features are 8 bytes of gate, up and each result.
template <int DT, uint32_t ACT, class L>
__device__ __forceinline__ void slope_few(const SlopeParams &p, const L &loop, const typename L::Acc &acc, int64_t p0, int64_t q0) {
#pragma unroll
    for (int j = 0; j < L::CB; ++j) {
        const int64_t row = q0 + loop.q_of(j);
#pragma unroll
        for (int i = 0; i < L::RB; ++i) {
            const int64_t col = p0 + loop.p_of(i, 0);
            if (row >= p.T || col >= p.F) continue;
            const Slopes s = slopes<DT, ACT>(*reinterpret_cast<const u32x2 *>(p.gate + row * p.ld_gate + col),
                                             *reinterpret_cast<const u32x2 *>(p.up + row * p.ld_up + col), acc.v[i][j]);
            const int64_t at = row * p.ld + col;
            store4<DT, true>(p.dg + at, p.part, s.dg);
            store4<DT, true>(p.du + at, p.part, s.du);
            store4<DT, true>(p.h + at, p.part, s.h);
        }
    }
}

template <int DT, class L>
__global__ __launch_bounds__(L::NT, 2) void ffn_slope(SlopeParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    loop.run_any(p.down, p0, p.dy, q0, p.H, 0, p.g.slabs, acc);
    if (!loop.active()) return;
    with_act(p.act, [&](auto A) {
        if constexpr (L::TQ <= LOSS_FEW) slope_few<DT, decltype(A)::value>(p, loop, acc, p0, q0);
        else slope_rows<DT, decltype(A)::value>(p, loop, acc, lds, p0, q0);
    });
}

// dx = dg . w_gate + du . w_up: one loop over both products' slabs, in `splits`
// slices of them.
struct SumParams {
    Matrix gate, up, dg, du;
    int F;
    Grid g;
    bool slots;
    void *out;
    int64_t ldo;
};
template <int DT, class L>
__global__ __launch_bounds__(L::NT, L::WAVES) void ffn_sum(SumParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    const int s0 = (int)((int64_t)p.g.slabs * split / p.g.splits), s1 = (int)((int64_t)p.g.slabs * (split + 1) / p.g.splits);
    loop.also(p.up, p0, p.du, q0, p.F);
    loop.run_any(p.gate, p0, p.dg, q0, p.F, s0, s1, acc);
    if (!p.slots) {
        store16<DT, true>(loop, acc, lds, static_cast<uint16_t *>(p.out), p.ldo, p0, q0, p.gate.rows, p.dg.rows);
        return;
    }
    if (!loop.active()) return;
    f32x4 *slot = slot_base<L>(static_cast<float *>(p.out), p.g, tp, tq, split, loop.wave, loop.lane);
#pragma unroll
    for (int i = 0; i < L::RB; ++i)
#pragma unroll
        for (int j = 0; j < L::CB; ++j) slot[(i * L::CB + j) * 64] = acc.v[i][j];
}

// The weights' gradients, each a product over the rows, in one launch: their tiles
// together fill the last round of workgroups better than three launches' (331 x 1536 x
// 4104: 31 us in three).
struct WeightParams {
    struct One {
        Matrix P, Q;
        Grid g;
        void *out;
        int64_t ldo;
        float *slots;   // g.splits > 1
        int end;        // the launch's workgroups up to and with this gradient's
    } one[3];
    int count, T, out_kind;
};
template <int DT, class L>
__global__ __launch_bounds__(L::NT, L::WAVES) void ffn_weights(WeightParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    int which = 0, start = 0;
    while (which + 1 < p.count && (int)blockIdx.x >= p.one[which].end) start = p.one[which++].end;
    const WeightParams::One &q = p.one[which];
    int tp, tq, split;
    place(q.g, q.end - start, (int)blockIdx.x - start, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    const int s0 = (int)((int64_t)q.g.slabs * split / q.g.splits), s1 = (int)((int64_t)q.g.slabs * (split + 1) / q.g.splits);
    loop.run_any(q.P, p0, q.Q, q0, p.T, s0, s1, acc);
    if (q.g.splits > 1) {
        f32x4 *slot = slot_base<L>(q.slots, q.g, tp, tq, split, loop.wave, loop.lane);
#pragma unroll
        for (int i = 0; i < L::RB; ++i)
#pragma unroll
            for (int j = 0; j < L::CB; ++j) slot[(i * L::CB + j) * 64] = acc.v[i][j];
        return;
    }
    if (p.out_kind == LO_16) {
        store16<DT, true>(loop, acc, lds, static_cast<uint16_t *>(q.out), q.ldo, p0, q0, q.P.rows, q.Q.rows);
        return;
    }
    const bool add = p.out_kind == LO_F32_ADD;
#pragma unroll
    for (int i = 0; i < L::RB; ++i) {
#pragma unroll
        for (int j = 0; j < L::CB; ++j) {
            const int64_t col = p0 + loop.p_of(i, 0), row = q0 + loop.q_of(j);
            if (row < q.Q.rows && col < q.P.rows) {
                f32x4 *at = reinterpret_cast<f32x4 *>(static_cast<float *>(q.out) + row * q.ldo + col);
                *at = add ? acc.v[i][j] + *at : acc.v[i][j];
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // one block row's loads in flight: no more registers are free
    }
}

// The slices' slots added in slice order; `end` counts blocks of 256 float4 here.
template <int DT, class L>
__global__ __launch_bounds__(256) void ffn_weights_join(WeightParams p) {
    constexpr int QUADS = L::TP * L::TQ / 4;
    int which = 0, start = 0;
    while (which + 1 < p.count && (int)blockIdx.x >= p.one[which].end) start = p.one[which++].end;
    const WeightParams::One &q = p.one[which];
    const int64_t id = ((int64_t)blockIdx.x - start) * 256 + threadIdx.x;
    const int tile = (int)(id / QUADS), f = (int)(id % QUADS);
    const int tp = tile % q.g.tiles_p, tq = tile / q.g.tiles_p;
    const int lane = f & 63, block = (f >> 6) % (L::RB * L::CB), wave = (f >> 6) / (L::RB * L::CB);
    const int i = block / L::CB, j = block % L::CB, wp = wave % L::WP, wq = wave / L::WP;
    const int64_t col = (int64_t)tp * L::TP + wp * L::WAVE_P + i * 16 + 4 * (lane >> 4);
    const int64_t row = (int64_t)tq * L::TQ + wq * L::WAVE_Q + j * 16 + (lane & 15);
    if (row >= q.Q.rows || col >= q.P.rows) return;
    const int64_t step = (int64_t)q.g.tiles_p * q.g.tiles_q * QUADS;
    const f32x4 *at = reinterpret_cast<const f32x4 *>(q.slots) + id;
    f32x4 v = at[0];
    int s = 1;
    for (; s + 4 <= q.g.splits; s += 4) {   // four loads in flight, added in order
        const f32x4 a = at[s * step], b = at[(s + 1) * step], c = at[(s + 2) * step], d = at[(s + 3) * step];
        v = (((v + a) + b) + c) + d;
    }
    for (; s < q.g.splits; ++s) v += at[s * step];
    const int64_t to = row * q.ldo + col;
    if (p.out_kind == LO_16) {
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(q.out) + to) = pack4<DT>(v);
        return;
    }
    f32x4 *out = reinterpret_cast<f32x4 *>(static_cast<float *>(q.out) + to);
    *out = p.out_kind == LO_F32_ADD ? v + *out : v;
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------
template <class L>
hipError_t run_gate(const FfnGate &a, void (*kernel)(GateParams), hipStream_t stream) {
    // a workgroup covers TP / 2 features: the grid is that of 2 F rows
    const GateParams q{matrix(a.gate), matrix(a.up), matrix(a.x), a.T, a.F, a.H, grid_of<L>(2 * (int64_t)a.F, a.T, a.H, 1), a.act,
                       a.h, a.kept_gate, a.kept_up, a.ldh, a.part, a.ld_gate, a.ld_up};
    hipLaunchKernelGGL(kernel, dim3(blocks_of(q.g)), dim3(L::NT), 0, stream, q);
    return hipGetLastError();
}
template <int DT, bool KC>
hipError_t gate(int tile, const FfnGate &a, hipStream_t stream) {
    using L128 = Loop<DT, KC, true, 128, 128, 2, 2, 3, 2, true>;
    using L256 = Loop<DT, KC, true, 256, 256, 2, 4, 3, 2, true>;
    if (tile == LT_128x128) return run_gate<L128>(a, ffn_gate<DT, L128>, stream);
    if (tile == LT_256x256) return run_gate<L256>(a, ffn_gate<DT, L256>, stream);
    if constexpr (KC) {   // halves of fewer than 64 rows: k contiguous only
        using F32 = ThinLoop<DT, true, true, 32, 32, 6, 1, true>;
        using F64 = ThinLoop<DT, true, true, 64, 64, 5, 1, true>;
        if (tile == LT_32x32) return run_gate<F32>(a, ffn_gate_few<DT, F32>, stream);
        if (tile == LT_64x64) return run_gate<F64>(a, ffn_gate_few<DT, F64>, stream);
    } else {
        using F128x32 = ThinLoop<DT, false, true, 128, 32, 4, 1, true>;
        using F128x64 = ThinLoop<DT, false, true, 128, 64, 3, 1, true>;
        if (tile == LT_128x32) return run_gate<F128x32>(a, ffn_gate_few<DT, F128x32>, stream);
        if (tile == LT_128x64) return run_gate<F128x64>(a, ffn_gate_few<DT, F128x64>, stream);
    }
    return hipErrorInvalidValue;
}

template <int DT, class L>
hipError_t run_slope(const FfnSlope &a, hipStream_t stream) {
    const SlopeParams q{matrix(a.down), matrix(a.dy), a.T, a.F, a.H, grid_of<L>(a.F, a.T, a.H, 1), a.act, a.gate, a.up,
                        a.ld_gate, a.ld_up, a.dg, a.du, a.h, a.ld, a.part};
    hipLaunchKernelGGL((ffn_slope<DT, L>), dim3(blocks_of(q.g)), dim3(L::NT), 0, stream, q);
    return hipGetLastError();
}
template <int DT, bool KC>
hipError_t slope(int tile, const FfnSlope &a, hipStream_t stream) {
    switch (tile) {
    case LT_128x128: return run_slope<DT, Loop<DT, KC, true, 128, 128, 2, 2, 3, 2>>(a, stream);
    case LT_256x256: return run_slope<DT, Loop<DT, KC, true, 256, 256, 2, 4, 3, 2>>(a, stream);
    case LT_64x64: return run_slope<DT, ThinLoop<DT, KC, true, 64, 64, 5>>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int DT, class L>
hipError_t run_sum(const FfnSum &a, hipStream_t stream) {
    SumParams q{matrix(a.gate), matrix(a.up), matrix(a.dg), matrix(a.du), a.F, grid_of<L>(a.gate.rows, a.dg.rows, a.F, a.splits),
                a.splits > 1, a.out, a.ldo};
    q.g.slabs *= 2;
    hipLaunchKernelGGL((ffn_sum<DT, L>), dim3(blocks_of(q.g)), dim3(L::NT), 0, stream, q);
    return hipGetLastError();
}
template <int DT, bool KC>
hipError_t sum(int tile, const FfnSum &a, hipStream_t stream) {
    switch (tile) {
    case LT_128x128: return run_sum<DT, Loop<DT, KC, true, 128, 128, 2, 2, KC ? 3 : 2, 2, false, 2>>(a, stream);
    case LT_256x256: return run_sum<DT, Loop<DT, KC, true, 256, 256, 2, 4, 3, 2, false, 2>>(a, stream);
    case LT_128x32: return run_sum<DT, ThinLoop<DT, KC, true, 128, 32, 4, 2, false, 2>>(a, stream);
    case LT_128x64: return run_sum<DT, ThinLoop<DT, KC, true, 128, 64, 3, 2, false, 2>>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int DT, int T>
hipError_t run_vec(const FfnGate &a, const LossMatrix &down, float *h, uint16_t *y, int64_t ldy, hipStream_t stream) {
    const GateParams q{matrix(a.gate), matrix(a.up), matrix(a.x), a.T, a.F, a.H, Grid{}, a.act,
                       nullptr, a.kept_gate, a.kept_up, 0, 0, a.ld_gate, a.ld_up};
    hipLaunchKernelGGL((ffn_gate_vec<DT, T>), dim3((unsigned)(a.F / 4)), dim3(256), 0, stream, q, h);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ffn_down_vec<DT, T>), dim3((unsigned)(down.rows / 4)), dim3(256), 0, stream, matrix(down), h, a.T, a.F, y, ldy);
    return hipGetLastError();
}

template <int DT, class L>
hipError_t run_weights(const FfnWeights &a, hipStream_t stream) {
    WeightParams q;
    q.count = 0;
    q.T = a.T;
    q.out_kind = a.out_kind;
    int end = 0;
    float *slots = a.slots;
    for (const FfnWeights::One &w : a.one) {
        if (!w.out) continue;
        const Grid g = grid_of<L>(w.P.rows, w.Q.rows, a.T, a.splits);
        end += (int)blocks_of(g);
        q.one[q.count++] = {matrix(w.P), matrix(w.Q), g, w.out, w.ldo, slots, end};
        if (slots) slots += (int64_t)blocks_of(g) * (L::TP * L::TQ);
    }
    if (!end) return hipSuccess;
    hipLaunchKernelGGL((ffn_weights<DT, L>), dim3((unsigned)end), dim3(L::NT), 0, stream, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    end = 0;
    for (int i = 0; i < q.count; ++i) q.one[i].end = end += q.one[i].g.tiles_p * q.one[i].g.tiles_q * (L::TP * L::TQ / 4 / 256);
    hipLaunchKernelGGL((ffn_weights_join<DT, L>), dim3((unsigned)end), dim3(256), 0, stream, q);
    return hipGetLastError();
}
template <int DT>
hipError_t weights(int tile, const FfnWeights &a, hipStream_t stream) {
    if (tile == LT_256x256) return run_weights<DT, Loop<DT, false, false, 256, 256, 2, 4, 2, 2>>(a, stream);
    if (tile == LT_128x128) return run_weights<DT, Loop<DT, false, false, 128, 128, 2, 2, 2, 2>>(a, stream);
    return hipErrorInvalidValue;
}

bool few(int tile) { return loss_tile_shape(tile).q <= LOSS_FEW; }

}  // namespace

hipError_t launch_ffn_gate(int dtype, int tile, const FfnGate &p, hipStream_t stream) {
    if (!p.x.kc || p.gate.kc != p.up.kc || few(tile) != (p.part > 0)) return hipErrorInvalidValue;
    if (p.gate.kc) return dtype == 0 ? gate<0, true>(tile, p, stream) : gate<1, true>(tile, p, stream);
    return dtype == 0 ? gate<0, false>(tile, p, stream) : gate<1, false>(tile, p, stream);
}

hipError_t launch_ffn_vec(int dtype, const FfnGate &p, const LossMatrix &down, float *h, uint16_t *y, int64_t ldy, hipStream_t stream) {
    if (!p.gate.kc || !p.up.kc || !down.kc || p.T > VEC_T || p.F % 8 || p.H % 8 || down.rows % 8) return hipErrorInvalidValue;
    if (p.T == 1) return dtype == 0 ? run_vec<0, 1>(p, down, h, y, ldy, stream) : run_vec<1, 1>(p, down, h, y, ldy, stream);
    if (p.T == 2) return dtype == 0 ? run_vec<0, 2>(p, down, h, y, ldy, stream) : run_vec<1, 2>(p, down, h, y, ldy, stream);
    return dtype == 0 ? run_vec<0, 4>(p, down, h, y, ldy, stream) : run_vec<1, 4>(p, down, h, y, ldy, stream);
}

hipError_t launch_ffn_sum(int dtype, int tile, const FfnSum &p, hipStream_t stream) {
    if (!p.dg.kc || !p.du.kc || p.gate.kc != p.up.kc || p.gate.ld != p.up.ld || p.dg.ld != p.du.ld || p.dg.part != p.du.part ||
        few(tile) != (p.dg.part > 0))
        return hipErrorInvalidValue;
    if (p.gate.kc) return dtype == 0 ? sum<0, true>(tile, p, stream) : sum<1, true>(tile, p, stream);
    return dtype == 0 ? sum<0, false>(tile, p, stream) : sum<1, false>(tile, p, stream);
}

hipError_t launch_ffn_weights(int dtype, int tile, const FfnWeights &p, hipStream_t stream) {
    if ((p.splits == 1) != (p.slots == nullptr)) return hipErrorInvalidValue;
    for (const FfnWeights::One &w : p.one)
        if (w.out && (w.P.kc || w.Q.kc)) return hipErrorInvalidValue;
    return dtype == 0 ? weights<0>(tile, p, stream) : weights<1>(tile, p, stream);
}

hipError_t launch_ffn_slope(int dtype, int tile, const FfnSlope &p, hipStream_t stream) {
    if (!p.dy.kc || few(tile) != (p.part > 0)) return hipErrorInvalidValue;
    if (p.down.kc) return dtype == 0 ? slope<0, true>(tile, p, stream) : slope<1, true>(tile, p, stream);
    return dtype == 0 ? slope<0, false>(tile, p, stream) : slope<1, false>(tile, p, stream);
}

}  // namespace dgw
