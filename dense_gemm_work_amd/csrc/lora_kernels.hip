// lora_kernels.hip -- gfx950 kernels of projections with low-rank adapters (gemm_lora.h).
//
// A row's adapter a adds (c_a x A_a^T) B_a^T to x W^T.  lora_low computes the narrow
// product c_a x A_a^T of a group of rows for each adapter that occurs in it; rows of
// other adapters are masked where they are loaded, so nothing is sorted or gathered.
// lora_product computes a tile of x W^T and goes on, in the same accumulators, over
// the adapters that occur among the tile's rows: their slabs of B against the
// narrow rows, again masked at the load.  Backward, the same two kernels with the
// factors' roles exchanged give dx; lora_outer sums the adapters' own gradients over
// their rows.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.h"
#include "tile.h"
#include "tile_store.h"

namespace dgw {

using namespace tile;

namespace {

constexpr int NONE = -1, BAD = -2;   // a row without an adapter, one whose adapter is out of range

__device__ __forceinline__ int adapter_of(const LoraRows &r, int64_t row) {
    if (row >= r.T) return NONE;
    const int64_t a = r.adapter[row];
    return a < 0 ? NONE : a < r.count ? (int)a : BAD;
}

// The adapters of TQ rows in LDS: each row's, and the distinct ones in the order of
// their first rows.
template <int TQ>
struct List {
    int id[TQ], of[TQ], count[TQ / 32 + 1];

    // Every thread of the workgroup calls this; it ends with a barrier.
    __device__ __forceinline__ void fill(const LoraRows &r, int64_t q0) {
        for (int t = threadIdx.x; t < TQ; t += blockDim.x) id[t] = adapter_of(r, q0 + t);
        __syncthreads();
        const int t = threadIdx.x, mine = t < TQ ? id[t] : NONE;
        bool first = mine >= 0;
        if (t < TQ)
            for (int u = 0; u < t && first; ++u) first = id[u] != mine;
        const uint64_t set = __ballot(first);
        if (t < TQ && (t & 63) == 0) count[t >> 6] = __popcll(set);
        __syncthreads();
        int at = __popcll(set & ((1ull << (t & 63)) - 1)), all = 0;
        for (int w = 0; w < (TQ + 63) / 64; ++w) {
            if (w < t >> 6) at += count[w];
            all += count[w];
        }
        if (first) of[at] = mine;
        __syncthreads();
        if (t == 0) count[TQ / 32] = all;
        __syncthreads();
    }
    __device__ __forceinline__ int n() const { return __builtin_amdgcn_readfirstlane(count[TQ / 32]); }
    __device__ __forceinline__ int adapter(int i) const { return __builtin_amdgcn_readfirstlane(of[i]); }
};

__device__ __forceinline__ Matrix shifted(Matrix m, int64_t elements) {
    m.base += elements;
    return m;
}

// ---------------------------------------------------------------------------
// The narrow products.
// ---------------------------------------------------------------------------
struct LowParams {
    LoraRows rows;
    Matrix f, x;
    int64_t stride;
    int R, K, slabs;
    int tiles_r, lists, splits;
    float *partial;
    uint16_t *low;
};

template <int DT, class L>
__global__ __launch_bounds__(L::NT, L::WAVES) void lora_low(LowParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    __shared__ List<L::TQ> list;
    int id = (int)blockIdx.x;
    const int split = id % p.splits;
    id /= p.splits;
    const int first = id % p.lists;
    id /= p.lists;
    const int64_t p0 = (int64_t)(id % p.tiles_r) * L::TP, q0 = (int64_t)(id / p.tiles_r) * L::TQ;
    list.fill(p.rows, q0);
    const int s0 = (int)((int64_t)p.slabs * split / p.splits), s1 = (int)((int64_t)p.slabs * (split + 1) / p.splits);
    L loop(lds);
    for (int i = first; i < list.n(); i += p.lists) {
        const int a = list.adapter(i);
        typename L::Acc acc;
        L::zero(acc);
        loop.run_any(shifted(p.f, a * p.stride), p0, p.x, q0, p.K, s0, s1, acc, [&](int r) { return list.id[r] == a; });
        if (!loop.active()) continue;
        const float scale = p.rows.scale ? p.rows.scale[a] : 1.0f;
#pragma unroll
        for (int b = 0; b < L::RB; ++b)
#pragma unroll
            for (int j = 0; j < L::CB; ++j) {
                const int col = (int)p0 + loop.p_of(b, 0);
                const int64_t row = q0 + loop.q_of(j);
                if (col >= p.R || list.id[loop.q_of(j)] != a) continue;
                const f32x4 v = acc.v[b][j];
                if (p.splits > 1)
                    *reinterpret_cast<f32x4 *>(p.partial + ((int64_t)split * p.rows.T + row) * p.R + col) = v;
                else
                    *reinterpret_cast<u32x2 *>(p.low + row * p.R + col) =
                        u32x2{pack2<DT>(v[0] * scale, v[1] * scale), pack2<DT>(v[2] * scale, v[3] * scale)};
            }
    }
}

// The slices' sums, added in slice order, scaled and rounded: a thread per four values.
template <int DT>
__global__ __launch_bounds__(256) void lora_low_join(LowParams p) {
    const int quads = p.R / 4;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, row = id / quads;
    if (row >= p.rows.T) return;
    const int a = adapter_of(p.rows, row);
    if (a < 0) return;
    const int col = 4 * (int)(id % quads);
    const f32x4 *at = reinterpret_cast<const f32x4 *>(p.partial + row * p.R + col);
    const int64_t step = (int64_t)p.rows.T * quads;
    f32x4 v = at[0];
    for (int s = 1; s < p.splits; ++s) v += at[s * step];
    const float scale = p.rows.scale ? p.rows.scale[a] : 1.0f;
    *reinterpret_cast<u32x2 *>(p.low + row * p.R + col) =
        u32x2{pack2<DT>(v[0] * scale, v[1] * scale), pack2<DT>(v[2] * scale, v[3] * scale)};
}

// ---------------------------------------------------------------------------
// The wide product and the adapters' part of it.
// ---------------------------------------------------------------------------
struct WideParams {
    LoraRows rows;
    Matrix P, x, f, low;
    int64_t stride;
    int K, R;
    Grid g;
    bool slots;
    void *out;
    int64_t ldo;
};

// acc += the products of the adapters' slabs (list entries from, from + every, ...)
// with the narrow rows, as a stream of (adapter, slab) items through NS stages.  Uses
// the first BYTES bytes of the LDS, which must be free, and leaves them free.
template <int DT, class L, int NS>
struct Extra {
    using OpP = typename L::OpP;
    using OpQ = typename L::OpQ;
    static constexpr int STAGE = OpP::SLAB + OpQ::SLAB, BYTES = NS * STAGE, LOADS = OpP::LOADS + OpQ::LOADS;
    static constexpr int PA = OpP::template addresses<L::RB>(), QA = OpQ::template addresses<L::CB>();
    static_assert((NS - 1) * LOADS < 64, "the wait counter holds the loads in flight");

    static __device__ __forceinline__ void run(const L &loop, const WideParams &p, int64_t p0, int64_t q0,
                                               const List<L::TQ> &list, int from, int every, typename L::Acc &acc) {
        const int lane = loop.lane, wave = loop.wave, slabs = (p.R + KB - 1) / KB;
        const int mine = list.n() > from ? (list.n() - from + every - 1) / every : 0, n = mine * slabs;
        if (!n) return;
        OpP P;
        OpQ Q;
        P.init(p.f, p0, p.R, wave, lane);
        Q.init(p.low, q0, p.R, wave, lane);
        int id[OpQ::LOADS];   // the adapters of the rows that this lane loads
#pragma unroll
        for (int x = 0; x < OpQ::LOADS; ++x) id[x] = list.id[8 * (wave * OpQ::LOADS + x) + (lane >> 3)];
        uint32_t pa[PA], qa[QA];
#pragma unroll
        for (int i = 0; i < PA; ++i) pa[i] = OpP::address(loop.lds0, loop.wp * L::WAVE_P, lane, i);
#pragma unroll
        for (int i = 0; i < QA; ++i) qa[i] = OpQ::address(loop.lds0 + OpP::SLAB, loop.wq * L::WAVE_Q, lane, i);
        int slab = 0, at = from;   // of the next item
        auto issue = [&](int stage) {
            const int a = list.adapter(at), s = slab;
            const uint32_t dst = loop.lds0 + stage * STAGE;
            const i32x4 rp = P.rsrc(s, a * p.stride * 2), rq = Q.rsrc(s);
#pragma unroll
            for (int x = 0; x < OpP::LOADS; ++x) P.template load<true>(rp, s, x, dst + wave * OpP::LOADS * 1024);
            const bool in = s * KB + Q.kc < p.R;
#pragma unroll
            for (int x = 0; x < OpQ::LOADS; ++x)
                load_lds16(rq, dst + OpP::SLAB + (wave * OpQ::LOADS + x) * 1024, in && id[x] == a ? Q.off[x] : OOB);
            if (++slab == slabs) {
                slab = 0;
                at += every;
            }
        };
        for (int i = 0; i < min(NS, n); ++i) issue(i);
        int st = 0;
        for (int i = 0; i < n; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            wait_stages<LOADS>(min(NS, n - i) - 1);
            barrier();
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t o = st * STAGE;
#pragma unroll
            for (int step = 0; step < 2; ++step) {
                u32x4 q[L::CB];
#pragma unroll
                for (int j = 0; j < L::CB; ++j) q[j] = OpQ::fragment(qa[OpQ::which(j, step)] + o + OpQ::constant(j, step));
#pragma unroll
                for (int b = 0; b < L::RB; ++b) {
                    const u32x4 f = OpP::fragment(pa[OpP::which(b, step)] + o + OpP::constant(b, step));
#pragma unroll
                    for (int j = 0; j < L::CB; ++j) acc.v[b][j] = mfma<DT>(f, q[j], acc.v[b][j]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            wait_lds();
            barrier();   // every wave has read the stage
            __builtin_amdgcn_sched_barrier(0);
            if (i + NS < n) issue(st);
            st = st + 1 == NS ? 0 : st + 1;
        }
        __syncthreads();
    }
    // This wave's LDS operations; its loads go on.
    static __device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt((15 | (3 << 14)) | (7 << 4)); }
};

template <int DT, class L, int NS>
__global__ __launch_bounds__(L::NT, 2) void lora_product(WideParams p) {
    using X = Extra<DT, L, NS>;
    constexpr int AT = (X::BYTES + 15) & ~15, NEED = AT + (int)sizeof(List<L::TQ>);
    constexpr int BYTES = NEED > L::LDS_BYTES ? NEED : L::LDS_BYTES;
    __shared__ __attribute__((aligned(16))) char lds[BYTES];
    int tp, tq, split;
    place(p.g, tp, tq, split);
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    const int s0 = (int)((int64_t)p.g.slabs * split / p.g.splits), s1 = (int)((int64_t)p.g.slabs * (split + 1) / p.g.splits);
    loop.run_any(p.P, p0, p.x, q0, p.K, s0, s1, acc);
    List<L::TQ> &list = *reinterpret_cast<List<L::TQ> *>(lds + AT);
    list.fill(p.rows, q0);
    X::run(loop, p, p0, q0, list, split, p.g.splits, acc);
#pragma unroll
    for (int j = 0; j < L::CB; ++j)
        if (list.id[loop.q_of(j)] == BAD)
#pragma unroll
            for (int i = 0; i < L::RB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.v[i][j][e] = __builtin_nanf("");
    if (!p.slots) {
        __syncthreads();
        store16<DT, true>(loop, acc, lds, static_cast<uint16_t *>(p.out), p.ldo, p0, q0, p.P.rows, p.x.rows);
        return;
    }
    if (!loop.active()) return;
    f32x4 *slot = slot_base<L>(static_cast<float *>(p.out), p.g, tp, tq, split, loop.wave, loop.lane);
#pragma unroll
    for (int i = 0; i < L::RB; ++i)
#pragma unroll
        for (int j = 0; j < L::CB; ++j) slot[(i * L::CB + j) * 64] = acc.v[i][j];
}

// The slices' slots added in slice order.
template <int DT, class L>
__global__ __launch_bounds__(256) void lora_join(WideParams p, const float *slots) {
    constexpr int QUADS = L::TP * L::TQ / 4;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= (int64_t)p.g.tiles_p * p.g.tiles_q * QUADS) return;
    const int tile = (int)(id / QUADS), f = (int)(id % QUADS);
    const int tp = tile % p.g.tiles_p, tq = tile / p.g.tiles_p;
    const int lane = f & 63, block = (f >> 6) % (L::RB * L::CB), wave = (f >> 6) / (L::RB * L::CB);
    const int i = block / L::CB, j = block % L::CB, wp = wave % L::WP, wq = wave / L::WP;
    const int64_t col = (int64_t)tp * L::TP + wp * L::WAVE_P + i * 16 + 4 * (lane >> 4);
    const int64_t row = (int64_t)tq * L::TQ + wq * L::WAVE_Q + j * 16 + (lane & 15);
    if (row >= p.x.rows || col >= p.P.rows) return;
    const int64_t step = (int64_t)p.g.tiles_p * p.g.tiles_q * QUADS;
    const f32x4 *at = reinterpret_cast<const f32x4 *>(slots) + id;
    f32x4 v = at[0];
    int s = 1;
    for (; s + 4 <= p.g.splits; s += 4) {   // four loads in flight, added in order
        const f32x4 a = at[s * step], b = at[(s + 1) * step], c = at[(s + 2) * step], d = at[(s + 3) * step];
        v = (((v + a) + b) + c) + d;
    }
    for (; s < p.g.splits; ++s) v += at[s * step];
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + row * p.ldo + col) =
        u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

// ---------------------------------------------------------------------------
// The adapters' own gradients.
// ---------------------------------------------------------------------------
// One wave per 64 rows.
__global__ __launch_bounds__(256) void lora_masks(LoraRows r, int64_t slabs, uint64_t *masks) {
    const int lane = threadIdx.x & 63;
    const int64_t slab = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (slab >= slabs) return;
    const int id = adapter_of(r, slab * 64 + lane);
    for (int a0 = 0; a0 < r.count; a0 += 64) {
        uint64_t keep = 0;
        for (int a = 0; a < min(64, r.count - a0); ++a) {
            const uint64_t m = __ballot(id == a0 + a);
            if (lane == a) keep = m;
        }
        if (a0 + lane < r.count) masks[(int64_t)(a0 + lane) * slabs + slab] = keep;
    }
}

struct OuterParams {
    Matrix P, Q;
    int T, slabs, count;
    const uint64_t *masks;
    int tiles_p, tiles_q, splits;
    float *partial;
    int out_kind;
    void *out;
    int64_t ldo, stride;
};

// Which slabs of [s0, s1) hold rows of an adapter, 64 slabs' masks at a time: lane l
// holds that of slab base + l.
struct Slabs {
    const uint64_t *masks;
    int base, end, lane;
    uint64_t own, left;
    __device__ __forceinline__ Slabs(const uint64_t *m, int s0, int s1, int lane_) : masks(m), base(s0), end(s1), lane(lane_) { load(); }
    __device__ __forceinline__ void load() {
        own = base + lane < end ? masks[base + lane] : 0;
        left = __ballot(own != 0);
    }
    // The next such slab and its mask; false behind the last.
    __device__ __forceinline__ bool next(int &slab, uint64_t &mask) {
        while (!left) {
            base += 64;
            if (base >= end) return false;
            load();
        }
        const int bit = __builtin_ctzll(left);
        left &= left - 1;
        slab = base + bit;
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)own, bit), hi = __builtin_amdgcn_readlane((int)(uint32_t)(own >> 32), bit);
        mask = (uint64_t)hi << 32 | lo;
        return true;
    }
};

template <int DT, int TP, int TQ>
__global__ __launch_bounds__(256) void lora_outer(OuterParams p) {
    constexpr int NS = 3, WP = TP / 32 > 2 ? 2 : 1, WQ = 4 / WP, RB = TP / WP / 16, CB = TQ / WQ / 16;
    using OpP = Operand<false, TP, 4>;
    using OpQ = Operand<false, TQ, 4>;
    constexpr int STAGE = OpP::SLAB + OpQ::SLAB, LOADS = OpP::LOADS + OpQ::LOADS;
    __shared__ __attribute__((aligned(16))) char lds[NS * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wp = wave % WP, wq = wave / WP;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
    int64_t id = blockIdx.x;
    const int tp = (int)(id % p.tiles_p);
    id /= p.tiles_p;
    const int tq = (int)(id % p.tiles_q);
    id /= p.tiles_q;
    const int split = (int)(id % p.splits);
    const int a = (int)(id / p.splits);
    const int64_t p0 = (int64_t)tp * TP, q0 = (int64_t)tq * TQ;
    OpP P;
    OpQ Q;
    P.init(p.P, p0, p.T, wave, lane);
    Q.init(p.Q, q0, p.T, wave, lane);
    uint32_t pa[RB], qa[CB];
#pragma unroll
    for (int i = 0; i < RB; ++i) pa[i] = OpP::address(lds0, wp * (TP / WP), lane, i);
#pragma unroll
    for (int i = 0; i < CB; ++i) qa[i] = OpQ::address(lds0 + OpP::SLAB, wq * (TQ / WQ), lane, i);
    const int s0 = (int)((int64_t)p.slabs * split / p.splits), s1 = (int)((int64_t)p.slabs * (split + 1) / p.splits);
    Slabs slabs(p.masks + (int64_t)a * p.slabs, s0, s1, lane);
    f32x4 acc[RB][CB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    bool more = true;
    int issued = 0;
    // rows of other adapters are masked in both operands: what they hold takes no part
    auto issue = [&](int stage) {
        int slab;
        uint64_t mask;
        if (!more || !(more = slabs.next(slab, mask))) return;
        ++issued;
        const uint32_t dst = lds0 + stage * STAGE;
        const i32x4 rp = P.rsrc(slab), rq = Q.rsrc(slab);
#pragma unroll
        for (int x = 0; x < OpP::LOADS; ++x) {
            const int k = (64 / (TP / 8)) * (wave * OpP::LOADS + x) + lane / (TP / 8);
            load_lds16(rp, dst + (wave * OpP::LOADS + x) * 1024, mask >> k & 1 ? P.off[x] : OOB);
        }
#pragma unroll
        for (int x = 0; x < OpQ::LOADS; ++x) {
            const int k = (64 / (TQ / 8)) * (wave * OpQ::LOADS + x) + lane / (TQ / 8);
            load_lds16(rq, dst + OpP::SLAB + (wave * OpQ::LOADS + x) * 1024, mask >> k & 1 ? Q.off[x] : OOB);
        }
    };
    for (int i = 0; i < NS; ++i) issue(i);
    int st = 0;
    for (int i = 0; i < issued; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        // a refill of the masks waits for everything; else this item's loads are done
        // once only the later items' are left
        wait_stages<LOADS>(issued - i - 1);
        barrier();
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t o = st * STAGE;
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            u32x4 q[CB];
#pragma unroll
            for (int j = 0; j < CB; ++j) q[j] = OpQ::fragment(qa[OpQ::which(j, step)] + o + OpQ::constant(j, step));
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                const u32x4 f = OpP::fragment(pa[OpP::which(b, step)] + o + OpP::constant(b, step));
#pragma unroll
                for (int j = 0; j < CB; ++j) acc[b][j] = mfma<DT>(f, q[j], acc[b][j]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((15 | (3 << 14)) | (7 << 4));   // this wave's LDS operations; its loads go on
        barrier();
        __builtin_amdgcn_sched_barrier(0);
        issue(st);
        st = st + 1 == NS ? 0 : st + 1;
    }
    const bool direct = p.splits == 1;
    const int64_t ldo = direct ? p.ldo : p.P.rows;
    const int64_t base = direct ? a * p.stride : ((int64_t)split * p.count + a) * p.Q.rows * p.P.rows;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int64_t col = p0 + wp * (TP / WP) + i * 16 + 4 * (lane >> 4), row = q0 + wq * (TQ / WQ) + j * 16 + (lane & 15);
            if (col >= p.P.rows || row >= p.Q.rows) continue;
            const int64_t at = base + row * ldo + col;
            f32x4 v = acc[i][j];
            if (!direct) {
                *reinterpret_cast<f32x4 *>(p.partial + at) = v;
            } else if (p.out_kind == LO_16) {
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + at) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
            } else {
                f32x4 *to = reinterpret_cast<f32x4 *>(static_cast<float *>(p.out) + at);
                if (p.out_kind == LO_F32_ADD) v += *to;
                *to = v;
            }
        }
}

template <int DT>
__global__ __launch_bounds__(256) void lora_outer_join(OuterParams p) {
    const int64_t quads = p.P.rows / 4, all = (int64_t)p.count * p.Q.rows * quads;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= all) return;
    const int64_t col = id % quads * 4, row = id / quads % p.Q.rows, a = id / quads / p.Q.rows;
    const f32x4 *from = reinterpret_cast<const f32x4 *>(p.partial) + id;
    f32x4 v = from[0];
    for (int s = 1; s < p.splits; ++s) v += from[s * all];
    const int64_t at = a * p.stride + row * p.ldo + col;
    if (p.out_kind == LO_16) {
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + at) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        return;
    }
    f32x4 *to = reinterpret_cast<f32x4 *>(static_cast<float *>(p.out) + at);
    if (p.out_kind == LO_F32_ADD) v += *to;
    *to = v;
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------
template <int DT, class L>
hipError_t run_low(const LoraLow &a, hipStream_t stream) {
    const LowParams q{a.rows, matrix(a.f.first), matrix(a.x), a.f.stride, a.R, a.K, (a.K + KB - 1) / KB,
                      (a.R + L::TP - 1) / L::TP, a.lists, a.splits, a.partial, a.low};
    const int64_t groups = ((int64_t)a.rows.T + L::TQ - 1) / L::TQ;
    hipLaunchKernelGGL((lora_low<DT, L>), dim3((unsigned)(groups * q.tiles_r * a.lists * a.splits)), dim3(L::NT), 0, stream, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t quads = (int64_t)a.rows.T * (a.R / 4);
    hipLaunchKernelGGL(lora_low_join<DT>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, q);
    return hipGetLastError();
}
template <int DT, bool KC>
hipError_t low(const LoraLow &a, hipStream_t stream) {
    switch (lora_low_tile(a.R, KC)) {
    case LL_64x64: return run_low<DT, ThinLoop<DT, KC, true, 64, 64, 5>>(a, stream);
    case LL_128x64: return run_low<DT, ThinLoop<DT, KC, true, 128, 64, 3>>(a, stream);
    default: break;
    }
    if constexpr (KC) return run_low<DT, ThinLoop<DT, true, true, 32, 64, 6>>(a, stream);
    return hipErrorInvalidValue;
}

template <class L>
WideParams wide_params(const LoraProduct &a) {
    LossMatrix low;
    low.base = a.low;
    low.ld = a.R;
    low.rows = a.rows.T;
    low.kc = true;
    return WideParams{a.rows, matrix(a.P), matrix(a.x), matrix(a.f.first), matrix(low), a.f.stride, a.K, a.R,
                      grid_of<L>(a.P.rows, a.x.rows, a.K, a.splits), a.splits > 1, a.out, a.ldo};
}

// f(loop type, stages of the adapters' slabs)
template <class L_, int DT_, int NS_>
struct Wide {
    using L = L_;
    static constexpr int DT = DT_, NS = NS_;
};
template <int DT, bool KC, class F>
hipError_t with_wide(int tile, F &&f) {
    switch (tile) {
    case LP_128x128: return f(Wide<Loop<DT, KC, true, 128, 128, 2, 2, KC ? 3 : 2, 2>, DT, 2>());
    case LP_256x256: return f(Wide<Loop<DT, KC, true, 256, 256, 2, 4, 3, 2>, DT, 2>());
    case LP_64x32: return f(Wide<ThinLoop<DT, KC, true, 64, 32, 6>, DT, 6>());
    case LP_64x64: return f(Wide<ThinLoop<DT, KC, true, 64, 64, 5>, DT, 4>());
    case LP_64x128: return f(Wide<ThinLoop<DT, KC, true, 64, 128, 3>, DT, 3>());
    default: return hipErrorInvalidValue;
    }
}
template <class F>
hipError_t with_wide(int dtype, int tile, bool kc, F &&f) {
    if (kc) return dtype == 0 ? with_wide<0, true>(tile, f) : with_wide<1, true>(tile, f);
    return dtype == 0 ? with_wide<0, false>(tile, f) : with_wide<1, false>(tile, f);
}

template <int DT, int TP, int TQ>
hipError_t run_outer(const LoraOuter &a, hipStream_t stream) {
    const OuterParams q{matrix(a.P), matrix(a.Q), a.T, (a.T + 63) / 64, a.count, a.masks, (a.P.rows + TP - 1) / TP,
                        (a.Q.rows + TQ - 1) / TQ, a.splits, a.partial, a.out_kind, a.out, a.ldo, a.stride};
    const int64_t blocks = (int64_t)a.count * q.tiles_p * q.tiles_q * a.splits;
    hipLaunchKernelGGL((lora_outer<DT, TP, TQ>), dim3((unsigned)blocks), dim3(256), 0, stream, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t quads = (int64_t)a.count * a.Q.rows * (a.P.rows / 4);
    hipLaunchKernelGGL(lora_outer_join<DT>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, q);
    return hipGetLastError();
}

}  // namespace

int lora_low_tile(int R, bool kc) { return R <= 32 && kc ? LL_32x64 : R <= 64 ? LL_64x64 : LL_128x64; }
int lora_low_rows(int tile) { return tile == LL_32x64 ? 32 : tile == LL_64x64 ? 64 : 128; }

hipError_t launch_lora_low(int dtype, const LoraLow &p, hipStream_t stream) {
    if (!p.x.kc) return hipErrorInvalidValue;
    if (p.f.first.kc) return dtype == 0 ? low<0, true>(p, stream) : low<1, true>(p, stream);
    return dtype == 0 ? low<0, false>(p, stream) : low<1, false>(p, stream);
}

LossTileShape lora_tile_shape(int tile) {
    if (tile == LP_64x32) return {64, 32, 2};
    return loss_tile_shape(tile);
}
int64_t lora_slots_bytes(int tile, int64_t rows_p, int64_t rows_q, int splits) {
    const LossTileShape s = lora_tile_shape(tile);
    return (rows_p + s.p - 1) / s.p * ((rows_q + s.q - 1) / s.q) * splits * (int64_t)s.p * s.q * 4;
}

hipError_t launch_lora_product(int dtype, int tile, const LoraProduct &p, hipStream_t stream) {
    if (!p.x.kc || p.P.kc != p.f.first.kc) return hipErrorInvalidValue;
    return with_wide(dtype, tile, p.P.kc, [&](auto w) {
        using W = decltype(w);
        const WideParams q = wide_params<typename W::L>(p);
        hipLaunchKernelGGL((lora_product<W::DT, typename W::L, W::NS>), dim3(blocks_of(q.g)), dim3(W::L::NT), 0, stream, q);
        return hipGetLastError();
    });
}
hipError_t launch_lora_join(int dtype, int tile, const LoraProduct &p, const float *slots, hipStream_t stream) {
    return with_wide(dtype, tile, true, [&](auto w) {   // the operands' storage does not matter here
        using W = decltype(w);
        const WideParams q = wide_params<typename W::L>(p);
        const int64_t quads = (int64_t)q.g.tiles_p * q.g.tiles_q * (W::L::TP * W::L::TQ / 4);
        hipLaunchKernelGGL((lora_join<W::DT, typename W::L>), dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream, q, slots);
        return hipGetLastError();
    });
}

hipError_t launch_lora_masks(const LoraRows &rows, uint64_t *masks, hipStream_t stream) {
    const int64_t slabs = ((int64_t)rows.T + 63) / 64;
    hipLaunchKernelGGL(lora_masks, dim3((unsigned)((slabs + 3) / 4)), dim3(256), 0, stream, rows, slabs, masks);
    return hipGetLastError();
}

hipError_t launch_lora_outer(int dtype, const LoraOuter &p, hipStream_t stream) {
    if (p.P.kc || p.Q.kc) return hipErrorInvalidValue;
    if (p.narrow_p) return dtype == 0 ? run_outer<0, 64, 128>(p, stream) : run_outer<1, 64, 128>(p, stream);
    return dtype == 0 ? run_outer<0, 128, 64>(p, stream) : run_outer<1, 128, 64>(p, stream);
}

}  // namespace dgw
