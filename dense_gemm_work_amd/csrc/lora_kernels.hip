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
#include <type_traits>

#include "lora.h"
#include "tile.h"
#include "tile_store.h"
#include "vec.h"

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
    static constexpr int WORDS = (TQ + 63) / 64;
    int id[TQ], of[TQ], count;

    // Every thread of the workgroup calls this, thread t with the adapter of row t; it
    // ends with a barrier.  One wave finds them, each step taking all rows of the first
    // row left: as many steps as adapters.  (Each row compared with all before it took
    // 6 us of a 128-row tile.)
    __device__ __forceinline__ void fill(int mine) {
        if (threadIdx.x < TQ) id[threadIdx.x] = mine;
        __syncthreads();
        if (threadIdx.x < 64) {
            int v[WORDS];
#pragma unroll
            for (int w = 0; w < WORDS; ++w) v[w] = 64 * w + threadIdx.x < TQ ? id[64 * w + threadIdx.x] : NONE;
            int n = 0;
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                for (uint64_t left = __ballot(v[w] >= 0); left; left = __ballot(v[w] >= 0)) {
                    const int a = __builtin_amdgcn_readlane(v[w], __builtin_ctzll(left));
#pragma unroll
                    for (int u = w; u < WORDS; ++u)
                        if (v[u] == a) v[u] = NONE;
                    if (threadIdx.x == 0) of[n] = a;
                    ++n;
                }
            if (threadIdx.x == 0) count = n;
        }
        __syncthreads();
    }
    __device__ __forceinline__ int n() const { return __builtin_amdgcn_readfirstlane(count); }
    __device__ __forceinline__ int adapter(int i) const { return __builtin_amdgcn_readfirstlane(of[i]); }
};

__device__ __forceinline__ Matrix shifted(Matrix m, int64_t elements) {
    m.base += elements;
    return m;
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt((15 | (3 << 14)) | (7 << 4)); }   // loads go on

// Sum over the slices of four values of a narrow row, in slice order, four loads in flight.
__device__ __forceinline__ f32x4 sum_slices(const float *at, int64_t step, int splits) {
    auto get = [&](int s) { return *reinterpret_cast<const f32x4 *>(at + s * step); };
    f32x4 v = get(0);
    int s = 1;
    for (; s + 4 <= splits; s += 4) {
        const f32x4 a = get(s), b = get(s + 1), c = get(s + 2), d = get(s + 3);
        v = (((v + a) + b) + c) + d;
    }
    for (; s < splits; ++s) v += get(s);
    return v;
}

// The same of eight.
__device__ __forceinline__ void sum_slices(const float *at, int64_t step, int splits, f32x4 &u, f32x4 &v) {
    auto get = [&](int s, int h) { return *reinterpret_cast<const f32x4 *>(at + s * step + 4 * h); };
    u = get(0, 0);
    v = get(0, 1);
    int s = 1;
    for (; s + 4 <= splits; s += 4) {
        f32x4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = get(s + i, 0);
            b[i] = get(s + i, 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u += a[i];
            v += b[i];
        }
    }
    for (; s < splits; ++s) {
        u += get(s, 0);
        v += get(s, 1);
    }
}

// ---------------------------------------------------------------------------
// The narrow products, unscaled, as fp32 slices [splits][T][R].  A workgroup takes
// one slice of k of a group of rows, and of the group's adapters every `lists`-th:
// those are the slowest part of its number, as most of them find no adapter and
// would leave their XCDs idle (8192 x 4096, rank 64: 57 us with them fastest).
// ---------------------------------------------------------------------------
struct LowParams {
    LoraRows rows;
    Matrix f, x;
    int64_t stride;
    int R, K, slabs;
    int tiles_r, groups, lists, splits;
    int blocks;
    float *partial;
};

template <class L>
__device__ __forceinline__ void low_block(const LowParams &p, int id, char *lds, List<L::TQ> &list) {
    const int split = id % p.splits;
    id /= p.splits;
    const int64_t p0 = (int64_t)(id % p.tiles_r) * L::TP;
    id /= p.tiles_r;
    const int64_t q0 = (int64_t)(id % p.groups) * L::TQ;
    const int first = id / p.groups;
    list.fill(adapter_of(p.rows, threadIdx.x < L::TQ ? q0 + threadIdx.x : p.rows.T));
    const int s0 = (int)((int64_t)p.slabs * split / p.splits), s1 = (int)((int64_t)p.slabs * (split + 1) / p.splits);
    L loop(lds);
    for (int i = first; i < list.n(); i += p.lists) {
        const int a = list.adapter(i);
        typename L::Acc acc;
        L::zero(acc);
        loop.run_any(shifted(p.f, a * p.stride), p0, p.x, q0, p.K, s0, s1, acc, [&](int r) { return list.id[r] == a; });
        if (!loop.active()) continue;
#pragma unroll
        for (int b = 0; b < L::RB; ++b)
#pragma unroll
            for (int j = 0; j < L::CB; ++j) {
                const int col = (int)p0 + loop.p_of(b, 0);
                const int64_t row = q0 + loop.q_of(j);
                if (col < p.R && list.id[loop.q_of(j)] == a)
                    *reinterpret_cast<f32x4 *>(p.partial + ((int64_t)split * p.rows.T + row) * p.R + col) = acc.v[b][j];
            }
    }
}

// Waves resident per SIMD of a workgroup of four with `bytes` of LDS for its tiles and a list.
// The list makes 64 x 64 tiles of five stages, half of a CU's LDS, one workgroup a CU.
constexpr int waves_with_list(int bytes) { return 2 * (bytes + (int)sizeof(List<64>)) <= 160 * 1024 ? 2 : 1; }

template <class L>
__global__ __launch_bounds__(L::NT, waves_with_list(L::LDS_BYTES)) void lora_low(LowParams p) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES];
    __shared__ List<L::TQ> list;
    low_block<L>(p, (int)blockIdx.x, lds, list);
}

// Few rows, many of them with an adapter of their own: a workgroup for a row and eight
// ranks, straight from memory, as one slice.  (Where the factor's rows are contiguous a
// wave reads 16 bytes of each: with up to 64 bytes, and as many fewer workgroups, the
// gradients' call for 96 x 4096 x 4096 with 64 adapters of rank 16 takes 54 us, not 46.)
template <int DT_, bool KC>
struct RowLow {
    static constexpr int DT = DT_, TP = 8, TQ = 64, NT = 256, LDS_BYTES = 4 * 8 * 4;
};
template <class L>
struct IsRowLow : std::false_type {};
template <int DT, bool KC>
struct IsRowLow<RowLow<DT, KC>> : std::true_type {};

template <int DT, bool KC>
__device__ __forceinline__ void row_block(const LowParams &p, int id, char *lds, RowLow<DT, KC>) {
    const int64_t t = id / p.tiles_r;
    const int r0 = id % p.tiles_r * 8, a = adapter_of(p.rows, t);
    if (a < 0) return;
    const uint16_t *f = p.f.base + a * p.stride, *x = p.x.base + t * p.x.ld;
    float(&red)[4][8][1] = *reinterpret_cast<float(*)[4][8][1]>(lds);
    if constexpr (KC) {
        const uint16_t *w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = f + (r0 + i) * p.f.ld;
        dot_rows<DT>(w, Rows16<DT>{x, 0}, 1, p.K, red);
    } else {
        float acc[8] = {};
#pragma unroll 4
        for (int k = threadIdx.x; k < p.K; k += 256) {
            const f32x8 v = unpack8<DT>(*reinterpret_cast<const u32x4 *>(f + k * p.f.ld + r0));
            float lo, hi;
            unpack2<DT>(x[k], lo, hi);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(v.v[e], lo, acc[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int o = 32; o; o >>= 1) acc[e] += __shfl_xor(acc[e], o);
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][e][0] = acc[e];
        }
        __syncthreads();
    }
    if (threadIdx.x < 8) p.partial[t * p.R + r0 + threadIdx.x] = joined(red, threadIdx.x, 0);
}

template <class L>
__device__ __forceinline__ void narrow_block(const LowParams &p, int id, char *lds, List<L::TQ> &list) {
    if constexpr (IsRowLow<L>::value) row_block(p, id, lds, L());
    else low_block<L>(p, id, lds, list);
}

// Which rows of each 64 have which adapter: one wave per 64 rows.
__device__ __forceinline__ void mask_block(const LoraRows &r, int id, uint64_t *masks) {
    const int lane = threadIdx.x & 63, slabs = (r.T + 63) / 64;
    const int slab = id * 4 + (threadIdx.x >> 6);
    if (slab >= slabs) return;
    const int mine = adapter_of(r, slab * (int64_t)64 + lane);
    for (int a0 = 0; a0 < r.count; a0 += 64) {
        uint64_t keep = 0;
        for (int a = 0; a < min(64, r.count - a0); ++a) {
            const uint64_t m = __ballot(mine == a0 + a);
            if (lane == a) keep = m;
        }
        if (a0 + lane < r.count) masks[(int64_t)(a0 + lane) * slabs + slab] = keep;
    }
}

// Backward: both narrow products (one factor has k contiguous, the other its rows) and
// the rows' masks in one launch.
template <class LK, class LR>
__global__ __launch_bounds__(256, waves_with_list(LK::LDS_BYTES > LR::LDS_BYTES ? LK::LDS_BYTES : LR::LDS_BYTES)) void lora_lows(LowParams k, LowParams r, uint64_t *masks) {
    __shared__ __attribute__((aligned(16))) char lds[LK::LDS_BYTES > LR::LDS_BYTES ? LK::LDS_BYTES : LR::LDS_BYTES];
    __shared__ List<LK::TQ> list;
    static_assert(LK::TQ == LR::TQ && LK::NT == 256 && LR::NT == 256, "one list, one size of workgroup");
    const int id = (int)blockIdx.x;
    if (id < k.blocks) narrow_block<LK>(k, id, lds, list);
    else if (id < k.blocks + r.blocks) narrow_block<LR>(r, id - k.blocks, lds, list);
    else mask_block(k.rows, id - k.blocks - r.blocks, masks);
}

// s and ds as the type holds them, for the adapters' gradients, [T][R]: a thread per
// four values.  low == nullptr: not kept.  Rounded once, after the scale, as operands of
// matrix instructions: da and db are off by sqrt 2 times their own rounding (0.0023 of
// their norm in bf16, 0.0003 in fp16); a second part would double lora_outers' work.
struct LowJoin {
    LoraRows rows;
    int R;
    struct One {
        const float *partial;
        int splits;
        uint16_t *low;
    } one[2];
    int blocks;   // of 256 threads
};
template <int DT>
__device__ __forceinline__ void join_block(const LowJoin &p, int64_t id) {
    const int64_t each = (int64_t)p.rows.T * (p.R / 4);
    const bool second = id >= each;
    if (second) id -= each;
    if (id >= each) return;
    const LowJoin::One q = second ? p.one[1] : p.one[0];
    const int quads = p.R / 4, col = 4 * (int)(id % quads);
    const int64_t row = id / quads;
    const int a = adapter_of(p.rows, row);
    if (a < 0 || !q.low) return;
    const float scale = p.rows.scale ? p.rows.scale[a] : 1.0f;
    const f32x4 v = sum_slices(q.partial + row * p.R + col, (int64_t)p.rows.T * p.R, q.splits) * scale;
    *reinterpret_cast<u32x2 *>(q.low + row * p.R + col) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}
template <int DT>
__global__ __launch_bounds__(256) void lora_low_join(LowJoin p) {
    join_block<DT>(p, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// The wide product and the adapters' part of it.
// ---------------------------------------------------------------------------
struct WideParams {
    LoraRows rows;
    Matrix P, x, f;
    int64_t stride;
    const float *partial;   // the narrow product's slices
    int low_splits;
    int K, R;
    Grid g;       // splits: slices of each of the tail's tiles
    int whole;    // tiles before the tail
    float *slots;   // the tail's slices
    void *out;
    int64_t ldo;
    LowJoin join;   // of the workgroups behind those of tiles
};
// Tiles that fill whole rounds of workgroups are computed whole, those of the last round
// (the tail: ids from `whole` on) in slices, so that they fill it too.
__host__ __device__ inline int wide_blocks(const Grid &g, int whole) { return whole + (g.tiles_p * g.tiles_q - whole) * g.splits; }
// The workgroup's tile, slice and, of a tail tile, number in the tail (else -1).
__device__ __forceinline__ int place_wide(const Grid &g, int whole, int b, int &tp, int &tq, int &split) {
    const int rest = g.tiles_p * g.tiles_q - whole;
    int id;
    split = 0;
    if (b < whole) {
        id = spread(whole, b);
    } else {
        id = spread(rest * g.splits, b - whole);
        split = id / rest;
        id = whole + id - split * rest;
    }
    tile_of(g, id, tp, tq);
    return b < whole ? -1 : id - whole;
}

// acc += the products of the adapters' slabs (list entries from, from + every, ...)
// with the narrow rows.  Those of the tile, 64 ranks at a time, are put together from
// their slices, scaled, rounded and laid down in LDS, and stay in registers; the
// adapters' slabs stream through NS stages, and each meets the 16-row blocks that hold
// rows of its own; what it holds reaches no other row.  Uses the first BYTES bytes of the
// LDS, which must be free, and leaves them free.
// s and ds are rounded once, after the scale, as operands of matrix instructions, which
// counts as much as the adapters' part of y and dx does: 0.00022 of y's norm, 0.00021 its own
// rounding (5000 x 4096 x 8192 fp16, 24 of rank 64), 0.0018 of dx's, 0.0017 its own (8192 x
// 4096 x 4096 bf16, eight of rank 64).  A second part would double the adapters' products.
// Few rows' join takes them unrounded.
template <int DT, class L, int NS>
struct Extra {
    using OpP = typename L::OpP;
    using OpQ = typename L::OpQ;
    static constexpr int STAGE = OpP::SLAB, LOADS = OpP::LOADS, ROWS_AT = NS * STAGE, BYTES = ROWS_AT + L::TQ * 128;
    static constexpr int PA = OpP::template addresses<L::RB>();
    static_assert((NS - 1) * LOADS < 64 && NS <= 8, "the wait counter holds the loads in flight");

    // Small tiles keep the narrow rows in registers, skip blocks without rows of the adapter
    // and keep a product for the rows of the adapter alone.  In the large ones any of these
    // spills accumulators (the last 100 to 180 registers of 256 x 256), and the others' rows
    // are multiplied as zeros, which an infinity or NaN of the adapter would carry into them:
    // where the sums hold one, they are made again with `scrub`, the finite part as before and
    // the rest added to the adapter's own rows.  (That the sums are looked at: 331.5 us instead
    // of 331 at 5000 x 4096 x 8192, 24 of rank 64; 118.6 instead of 113.9 at 1000 x 2048 x 4096
    // with 64 of rank 16 mixed row by row.  One broken adapter: 1160 and 340 us; a broken row of
    // x: 325 and 178.)
    static constexpr bool HOLD = L::RB * L::CB <= 8, KC = OpP::which(1, 0) == 0;
    static __device__ __forceinline__ bool nonfinite(uint32_t v) {
        constexpr uint32_t EXPONENT = DT == 0 ? 0x7f80u : 0x7c00u;
        return (v & EXPONENT) == EXPONENT;
    }
    static __device__ __forceinline__ u32x4 masked(u32x4 v, bool keep) {
        return u32x4{keep ? v[0] : 0u, keep ? v[1] : 0u, keep ? v[2] : 0u, keep ? v[3] : 0u};
    }
    // scrub: an adapter's slab without its infinities and NaN, and whether the thread saw any.
    // Between barriers.
    static __device__ __forceinline__ bool clear_nonfinite(char *stage) {
        bool any = false;
        for (int f = threadIdx.x; f < STAGE / 16; f += L::NT) {
            u32x4 v = *reinterpret_cast<u32x4 *>(stage + 16 * f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                any |= nonfinite(v[i]) || nonfinite(v[i] >> 16);
                v[i] &= (nonfinite(v[i]) ? 0u : 0xffffu) | (nonfinite(v[i] >> 16) ? 0u : 0xffff0000u);
            }
            *reinterpret_cast<u32x4 *>(stage + 16 * f) = v;
        }
        __syncthreads();
        return any;
    }
    // scrub: what the slab's infinities and NaN add to the rows of their own adapter (a slice
    // adds those of every adapter: twice is the same).
    static __device__ __forceinline__ void add_nonfinite(const L &loop, const char *rows, const WideParams &p, int64_t p0, int slab,
                                                         const int (&id)[L::CB], typename L::Acc &acc) {
        const int ranks = min(KB, p.R - slab * KB);
#pragma unroll
        for (int j = 0; j < L::CB; ++j) {
            if (id[j] < 0) continue;
            const uint16_t *f = p.f.base + id[j] * p.stride + (KC ? p0 * p.f.ld : p0) + (int64_t)slab * KB * (KC ? 1 : p.f.ld);
            const char *own = rows + loop.q_of(j) * 128;
#pragma unroll 1
            for (int r = 0; r < ranks; ++r) {
                const uint32_t word = *reinterpret_cast<const uint16_t *>(own + (((r >> 3) ^ swz_kc(loop.q_of(j))) << 4) + (r & 7) * 2);
                float s, none;
                unpack2<DT>(word, s, none);
                int ld = (int)p.f.ld;
                asm volatile("" : "+s"(ld));   // or the offsets of every block would be kept in registers
#pragma unroll
                for (int b = 0; b < L::RB; ++b) {
                    const int row = loop.p_of(b, 0);
                    if (p0 + row < p.f.rows)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = f[KC ? (row + e) * ld : row + e];
                            float v;
                            unpack2<DT>(w, v, none);
                            if (nonfinite(w)) acc.v[b][j][e] = __builtin_fmaf(v, s, acc.v[b][j][e]);
                        }
                    __builtin_amdgcn_sched_barrier(0);
                }
                f += KC ? 1 : ld;
            }
        }
    }
    // Whether any thread of the workgroup says so.  The LDS is free, before and after.
    static __device__ __forceinline__ bool any_thread(bool mine, char *lds) {
        int *flag = reinterpret_cast<int *>(lds);
        if (threadIdx.x == 0) *flag = 0;
        __syncthreads();
        if (mine) *flag = 1;
        __syncthreads();
        const bool any = __builtin_amdgcn_readfirstlane(*flag);
        __syncthreads();
        return any;
    }
    // Whether a sum of the workgroup's is infinite or NaN.
    static __device__ __forceinline__ bool any_nonfinite(const typename L::Acc &acc, char *lds) {
        float zero = 0.0f;
#pragma unroll
        for (int b = 0; b < L::RB; ++b)
#pragma unroll
            for (int j = 0; j < L::CB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) zero = __builtin_fmaf(acc.v[b][j][e], 0.0f, zero);
        return any_thread(zero != 0.0f, lds);
    }

    static __device__ __forceinline__ void run(const L &loop, char *lds, const WideParams &p, int64_t p0, int64_t q0,
                                               const List<L::TQ> &list, int from, int every, bool scrub, typename L::Acc &acc) {
        const int lane = loop.lane, wave = loop.wave, slabs = (p.R + KB - 1) / KB;
        const int n = list.n() > from ? (list.n() - from + every - 1) / every : 0;
        if (!n) {
            __syncthreads();   // the list is read: its LDS is free, too
            return;
        }
        OpP P;
        P.init(p.f, p0, p.R, wave, lane);
        int id[L::CB];   // the adapters of the rows that this lane multiplies
#pragma unroll
        for (int j = 0; j < L::CB; ++j) id[j] = list.id[loop.q_of(j)];
        uint32_t pa[PA];
#pragma unroll
        for (int i = 0; i < PA; ++i) pa[i] = OpP::address(loop.lds0, loop.wp * L::WAVE_P, lane, i);
#pragma unroll 1
        for (int slab = 0; slab < slabs; ++slab) {
            auto issue = [&](int i, int stage) {
                const i32x4 rp = P.rsrc(slab, list.adapter(from + i * every) * p.stride * 2);
#pragma unroll
                for (int x = 0; x < LOADS; ++x) P.template load<true>(rp, slab, x, loop.lds0 + (stage * STAGE + wave * LOADS * 1024));
            };
            for (int i = 0; i < min(NS, n); ++i) issue(i, i);
#pragma unroll 1
            for (int f = threadIdx.x; f < L::TQ * 8; f += L::NT) {
                const int r = f >> 3, c = f & 7, col = slab * KB + 8 * c, a = list.id[r];
                u32x4 w = u32x4{0u, 0u, 0u, 0u};
                if (a >= 0 && col < p.R) {
                    const float *at = p.partial + (q0 + r) * p.R + col, scale = p.rows.scale ? p.rows.scale[a] : 1.0f;
                    const int64_t step = (int64_t)p.rows.T * p.R;
                    f32x4 u, v;
                    sum_slices(at, step, p.low_splits, u, v);
                    u *= scale;
                    v *= scale;
                    w = u32x4{pack2<DT>(u[0], u[1]), pack2<DT>(u[2], u[3]), pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
                }
                *reinterpret_cast<u32x4 *>(lds + ROWS_AT + r * 128 + ((c ^ swz_kc(r)) << 4)) = w;
            }
            __syncthreads();
            auto narrow = [&](int step, int j) {
                return *reinterpret_cast<const u32x4 *>(lds + ROWS_AT + loop.q_of(j) * 128 +
                                                        (((4 * step + (lane >> 4)) ^ swz_kc(loop.q_of(j))) << 4));
            };
            u32x4 q[HOLD ? 2 : 1][L::CB];
            if constexpr (HOLD)
#pragma unroll
                for (int step = 0; step < 2; ++step)
#pragma unroll
                    for (int j = 0; j < L::CB; ++j) q[step][j] = narrow(step, j);
            int st = 0;
            bool cleared = false;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                wait_stages<LOADS>(min(NS, n - i) - 1);
                barrier();
                __builtin_amdgcn_sched_barrier(0);
                const uint32_t o = st * STAGE;
                const int a = list.adapter(from + i * every);
                if constexpr (HOLD) {
                    u32x4 f[2][L::RB];
#pragma unroll
                    for (int step = 0; step < 2; ++step)
#pragma unroll
                        for (int b = 0; b < L::RB; ++b) f[step][b] = OpP::fragment(pa[OpP::which(b, step)] + o + OpP::constant(b, step));
#pragma unroll
                    for (int j = 0; j < L::CB; ++j) {
                        if (!__any(id[j] == a)) continue;
#pragma unroll
                        for (int b = 0; b < L::RB; ++b) {
                            const f32x4 v = mfma<DT>(f[1][b], q[1][j], mfma<DT>(f[0][b], q[0][j], acc.v[b][j]));
                            acc.v[b][j] = id[j] == a ? v : acc.v[b][j];
                        }
                    }
                } else {
                    if (scrub) cleared |= clear_nonfinite(lds + o);
#pragma unroll
                    for (int step = 0; step < 2; ++step) {
#pragma unroll
                        for (int j = 0; j < L::CB; ++j) q[0][j] = masked(narrow(step, j), id[j] == a);
#pragma unroll
                        for (int b = 0; b < L::RB; ++b) {
                            const u32x4 f = OpP::fragment(pa[OpP::which(b, step)] + o + OpP::constant(b, step));
#pragma unroll
                            for (int j = 0; j < L::CB; ++j) acc.v[b][j] = mfma<DT>(f, q[0][j], acc.v[b][j]);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                wait_lds();
                barrier();   // every wave has read the stage
                __builtin_amdgcn_sched_barrier(0);
                if (i + NS < n) issue(i + NS, st);
                st = st + 1 == NS ? 0 : st + 1;
            }
            if constexpr (!HOLD)
                if (scrub && any_thread(cleared, lds)) {
                    add_nonfinite(loop, lds + ROWS_AT, p, p0, slab, id, acc);
                    __syncthreads();   // the rows have been read
                }
        }
        __syncthreads();
    }
};

// Slot of a tail tile's slice: a wave's blocks one after the other, each 64 float4.
template <class L>
__device__ __forceinline__ f32x4 *wide_slot(const WideParams &p, int tail, int split, int quad) {
    const int64_t rest = p.g.tiles_p * p.g.tiles_q - p.whole;
    return reinterpret_cast<f32x4 *>(p.slots) + (split * rest + tail) * (L::TP * L::TQ / 4) + quad;
}

template <int DT, class L, int NS>
__global__ __launch_bounds__(L::NT, 2) void lora_product(WideParams p) {
    using X = Extra<DT, L, NS>;
    constexpr int NEED = X::BYTES + (int)sizeof(List<L::TQ>);
    constexpr int BYTES = NEED > L::LDS_BYTES ? NEED : L::LDS_BYTES;
    __shared__ __attribute__((aligned(16))) char lds[BYTES];
    static_assert(L::NT >= L::TQ, "a thread for each row");
    const int wide = wide_blocks(p.g, p.whole);
    if ((int)blockIdx.x >= wide) {
        join_block<DT>(p.join, ((int64_t)blockIdx.x - wide) * L::NT + threadIdx.x);
        return;
    }
    int tp, tq, split;
    const int tail = place_wide(p.g, p.whole, (int)blockIdx.x, tp, tq, split), splits = tail < 0 ? 1 : p.g.splits;
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    const int mine = adapter_of(p.rows, threadIdx.x < L::TQ ? q0 + threadIdx.x : p.rows.T);
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    const int s0 = (int)((int64_t)p.g.slabs * split / splits), s1 = (int)((int64_t)p.g.slabs * (split + 1) / splits);
    List<L::TQ> &list = *reinterpret_cast<List<L::TQ> *>(lds + X::BYTES);
    // Small tiles: last, the rows' adapters on their way meanwhile.  Large ones: first, and
    // one form of the loop for every K: what lives across their loop, or accumulators
    // that meet two loops, spill hundreds of registers in its last iterations.
    if constexpr (X::HOLD) loop.run_any(p.P, p0, p.x, q0, p.K, s0, s1, acc);
    if (p.partial) {   // else the join adds the adapters
        list.fill(mine);
        X::run(loop, lds, p, p0, q0, list, split, splits, false, acc);
        if constexpr (!X::HOLD)
            if (list.n() > 0 && X::any_nonfinite(acc, lds)) {
                L::zero(acc);
                X::run(loop, lds, p, p0, q0, list, split, splits, true, acc);
            }
    }
    if constexpr (!X::HOLD) loop.template run<true>(p.P, p0, p.x, q0, p.K, s0, s1, acc);
#pragma unroll
    for (int j = 0; j < L::CB; ++j)
        if (p.partial && adapter_of(p.rows, q0 + loop.q_of(j)) == BAD)
#pragma unroll
            for (int i = 0; i < L::RB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.v[i][j][e] = __builtin_nanf("");
    if (tail < 0) {
        store16<DT, true>(loop, acc, lds, static_cast<uint16_t *>(p.out), p.ldo, p0, q0, p.P.rows, p.x.rows);
        return;
    }
    if (!loop.active()) return;
    f32x4 *slot = wide_slot<L>(p, tail, split, loop.wave * (L::RB * L::CB * 64) + loop.lane);
#pragma unroll
    for (int i = 0; i < L::RB; ++i)
#pragma unroll
        for (int j = 0; j < L::CB; ++j) slot[(i * L::CB + j) * 64] = acc.v[i][j];
}

// The tail's slots added in slice order, 256 float4 a block.
template <int DT, class L>
__device__ __forceinline__ void tail_block(const WideParams &p, int64_t id) {
    constexpr int QUADS = L::TP * L::TQ / 4;
    const int64_t rest = p.g.tiles_p * p.g.tiles_q - p.whole;
    const int tail = (int)(id / QUADS), f = (int)(id % QUADS);
    int tp, tq;
    tile_of(p.g, p.whole + tail, tp, tq);
    const int lane = f & 63, block = (f >> 6) % (L::RB * L::CB), wave = (f >> 6) / (L::RB * L::CB);
    const int i = block / L::CB, j = block % L::CB, wp = wave % L::WP, wq = wave / L::WP;
    const int64_t col = (int64_t)tp * L::TP + wp * L::WAVE_P + i * 16 + 4 * (lane >> 4);
    const int64_t row = (int64_t)tq * L::TQ + wq * L::WAVE_Q + j * 16 + (lane & 15);
    if (row >= p.x.rows || col >= p.P.rows) return;
    const f32x4 v = sum_slices(reinterpret_cast<const float *>(wide_slot<L>(p, tail, 0, f)), rest * (L::TP * L::TQ), p.g.splits);
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + row * p.ldo + col) =
        u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}
template <int DT, class L>
__global__ __launch_bounds__(256) void lora_join(WideParams p) {
    tail_block<DT, L>(p, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------
// Few rows of small ranks, each perhaps with an adapter of its own: the wide and the
// narrow product run side by side in one launch, and the join of the wide one's
// slices adds the adapters' part, row by row, in fp32.  (96 x 4096 x 4096, 64 adapters
// of rank 16: 21 us; the adapters in the product's tiles, after the narrow product's launch: 46.)
// ---------------------------------------------------------------------------
template <class L, class LN>
__global__ __launch_bounds__(256, waves_with_list(L::LDS_BYTES > LN::LDS_BYTES ? L::LDS_BYTES : LN::LDS_BYTES)) void lora_few(WideParams w, LowParams n, int wide) {
    __shared__ __attribute__((aligned(16))) char lds[L::LDS_BYTES > LN::LDS_BYTES ? L::LDS_BYTES : LN::LDS_BYTES];
    __shared__ List<LN::TQ> list;
    static_assert(L::NT == 256 && LN::NT == 256, "one size of workgroup");
    if ((int)blockIdx.x >= wide) {
        narrow_block<LN>(n, (int)blockIdx.x - wide, lds, list);
        return;
    }
    int tp, tq, split;
    const int tile = place_wide(w.g, 0, (int)blockIdx.x, tp, tq, split);   // every tile in slices
    const int64_t p0 = (int64_t)tp * L::TP, q0 = (int64_t)tq * L::TQ;
    L loop(lds);
    typename L::Acc acc;
    L::zero(acc);
    const int s0 = (int)((int64_t)w.g.slabs * split / w.g.splits), s1 = (int)((int64_t)w.g.slabs * (split + 1) / w.g.splits);
    loop.run_any(w.P, p0, w.x, q0, w.K, s0, s1, acc);
    if (!loop.active()) return;
    f32x4 *slot = wide_slot<L>(w, tile, split, loop.wave * (L::RB * L::CB * 64) + loop.lane);
#pragma unroll
    for (int j = 0; j < L::CB; ++j) {
        if (q0 + 16 * j >= w.x.rows) break;   // blocks of rows that are not there
#pragma unroll
        for (int i = 0; i < L::RB; ++i) slot[(i * L::CB + j) * 64] = acc.v[i][j];
    }
}

// At most VEC_T rows of x and w with k contiguous: the wide product by dot_rows, eight
// outputs a workgroup, into the slots of 64 x 32 tiles as one slice.
template <int DT, int T, class L, class LN>
__global__ __launch_bounds__(256) void lora_few_vec(WideParams w, LowParams n, int wide) {
    __shared__ __attribute__((aligned(16))) char lds[LN::LDS_BYTES];
    __shared__ List<LN::TQ> list;
    __shared__ float red[4][8][T];
    static_assert(LN::NT == 256 && L::TP == 64 && L::TQ == 32, "the join's tiles");
    if ((int)blockIdx.x >= wide) {
        narrow_block<LN>(n, (int)blockIdx.x - wide, lds, list);
        return;
    }
    const int o0 = (int)blockIdx.x * 8;
    const uint16_t *rows[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rows[i] = w.P.base + (int64_t)(o0 + i) * w.P.ld;
    dot_rows<DT>(rows, Rows16<DT>{w.x.base, w.x.ld}, w.x.rows, w.K, red);
    const int i = threadIdx.x & 7, t = threadIdx.x >> 3, o = o0 + i;
    if (t >= T || t >= w.x.rows) return;
    // one tile of rows, so tile ids along P: tile_of's bands hold whole columns
    float *slot = w.slots + (int64_t)(o >> 6) * (L::TP * L::TQ);
    slot[((o >> 4) & 3) * L::CB * 256 + (t + 16 * ((o >> 2) & 3)) * 4 + (o & 3)] = joined(red, i, t);
}

// A workgroup: 16 rows (block j of a tile of 64 x 16 cb) by the tile's 64 columns, a wave
// for each 16 of them.
constexpr int FEW_LDS = 16 * (LORA_FEW_R + 4);   // floats
template <int DT, bool KC>
__device__ __forceinline__ void few_join_block(const WideParams &p, int cb, int id, float *narrow) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = id % cb, tile = id / cb, floats_of_tile = 64 * 16 * cb;
    int tp, tq;
    tile_of(p.g, tile, tp, tq);
    const int64_t first = (int64_t)tq * 16 * cb + 16 * j, row = first + (lane & 15);
    const int64_t col = (int64_t)tp * 64 + 16 * wave + 4 * (lane >> 4);
    if (first >= p.x.rows) return;
    // the slices' sums first, whether or not their rows have adapters: no load waits for
    // another
    const int quads = p.R / 4, ld = p.R + 4;   // 4 floats of padding against bank conflicts
    const bool in = row < p.x.rows && col < p.P.rows;
    const int a = in ? adapter_of(p.rows, row) : NONE;
    f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
        const int64_t step = (int64_t)p.g.tiles_p * p.g.tiles_q * floats_of_tile;
        v = sum_slices(p.slots + tile * (int64_t)floats_of_tile + (wave * cb + j) * 256 + lane * 4, step, p.g.splits);
    }
    const float scale = a >= 0 && p.rows.scale ? p.rows.scale[a] : 1.0f;
    for (int f = threadIdx.x; f < 16 * quads; f += 256) {
        const int r = f / quads, q = f % quads;
        if (first + r < p.x.rows)
            *reinterpret_cast<f32x4 *>(narrow + r * ld + 4 * q) =
                sum_slices(p.partial + (first + r) * p.R + 4 * q, (int64_t)p.rows.T * p.R, p.low_splits);
    }
    __syncthreads();
    if (!in) return;
    if (a >= 0) {
        f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const float *s = narrow + (lane & 15) * ld;
        const uint16_t *f = p.f.base + a * p.stride;
        if constexpr (KC) {   // four rows of the factor, which lie one after the other
#pragma unroll 2
            for (int r = 0; r < p.R; r += 8) {
                const f32x4 s0 = *reinterpret_cast<const f32x4 *>(s + r), s1 = *reinterpret_cast<const f32x4 *>(s + r + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(f + (col + e) * p.f.ld + r);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        float lo, hi;
                        unpack2<DT>(w[h], lo, hi);
                        sum[e] = __builtin_fmaf(lo, h < 2 ? s0[2 * h] : s1[2 * h - 4], sum[e]);
                        sum[e] = __builtin_fmaf(hi, h < 2 ? s0[2 * h + 1] : s1[2 * h - 3], sum[e]);
                    }
                }
            }
        } else {
#pragma unroll 8
            for (int r = 0; r < p.R; ++r) {
                const f32x4 w = unpack4<DT>(*reinterpret_cast<const u32x2 *>(f + r * p.f.ld + col));
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(w[e], s[r], sum[e]);
            }
        }
        v += sum * scale;
    } else if (a == BAD) {
        v = f32x4{1.0f, 1.0f, 1.0f, 1.0f} * __builtin_nanf("");
    }
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + row * p.ldo + col) =
        u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

template <int DT, bool KC>
__global__ __launch_bounds__(256) void lora_few_join(WideParams p, int cb) {
    __shared__ __attribute__((aligned(16))) float narrow[FEW_LDS];
    few_join_block<DT, KC>(p, cb, (int)blockIdx.x, narrow);
}

// ---------------------------------------------------------------------------
// The adapters' own gradients.
// ---------------------------------------------------------------------------
struct OuterParams {
    Matrix P, Q;
    int T, slabs, count;
    const uint64_t *masks;
    int tiles_p, tiles_q, splits;
    int blocks;
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

template <int TP, int TQ, int NS = 3>
constexpr int outer_lds() { return NS * (TP + TQ) * KB * 2; }

// NS: stages.  Few rows have one or two slabs for each of their adapters: one stage, so that
// six workgroups fit a CU (96 x 4096 x 4096, 64 adapters of rank 16, with dx's join: 24 us, in
// three stages 31).
template <int DT, int TP, int TQ, int NS = 3>
__device__ __forceinline__ void outer_block(const OuterParams &p, int64_t id, char *lds) {
    constexpr int WP = TP / 32 > 2 ? 2 : 1, WQ = 4 / WP, RB = TP / WP / 16, CB = TQ / WQ / 16;
    using OpP = Operand<false, TP, 4>;
    using OpQ = Operand<false, TQ, 4>;
    constexpr int STAGE = OpP::SLAB + OpQ::SLAB, LOADS = OpP::LOADS + OpQ::LOADS;
    static_assert(NS * STAGE == outer_lds<TP, TQ, NS>(), "the stages");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wp = wave % WP, wq = wave / WP;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
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
        wait_lds();
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

// da and db: the wide side contiguous in one, the narrow side in the other.
template <int DT>
__global__ __launch_bounds__(256, 2) void lora_outers(OuterParams wide, OuterParams narrow) {
    __shared__ __attribute__((aligned(16))) char lds[outer_lds<128, 64>()];
    const int64_t id = blockIdx.x;
    if (id < wide.blocks) outer_block<DT, 128, 64>(wide, id, lds);
    else outer_block<DT, 64, 128>(narrow, id - wide.blocks, lds);
}
// The same, with the blocks that join dx's tail behind them.
template <int DT, class L>
__global__ __launch_bounds__(256, 2) void lora_join_outers(WideParams p, OuterParams wide, OuterParams narrow) {
    __shared__ __attribute__((aligned(16))) char lds[outer_lds<128, 64>()];
    const int64_t id = (int64_t)blockIdx.x - wide.blocks - narrow.blocks;
    if (id >= 0) tail_block<DT, L>(p, id * 256 + threadIdx.x);
    else if ((int)blockIdx.x < wide.blocks) outer_block<DT, 128, 64>(wide, blockIdx.x, lds);
    else outer_block<DT, 64, 128>(narrow, (int64_t)blockIdx.x - wide.blocks, lds);
}

// The slices of da and db added in slice order, a thread per four values: the first
// `wide_blocks` workgroups those of one, the others those of the other.
template <int DT>
__global__ __launch_bounds__(256) void lora_outer_join(OuterParams wide, OuterParams narrow, int wide_blocks) {
    const bool first = (int)blockIdx.x < wide_blocks;
    const OuterParams &p = first ? wide : narrow;
    const int64_t quads = p.P.rows / 4, all = (int64_t)p.count * p.Q.rows * quads;
    const int64_t id = (int64_t)(blockIdx.x - (first ? 0 : wide_blocks)) * 256 + threadIdx.x;
    if (id >= all) return;
    const int64_t col = id % quads * 4, row = id / quads % p.Q.rows, a = id / quads / p.Q.rows;
    f32x4 v = sum_slices(p.partial + id * 4, all * 4, p.splits);
    const int64_t at = a * p.stride + row * p.ldo + col;
    if (p.out_kind == LO_16) {
        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p.out) + at) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        return;
    }
    f32x4 *to = reinterpret_cast<f32x4 *>(static_cast<float *>(p.out) + at);
    if (p.out_kind == LO_F32_ADD) v += *to;
    *to = v;
}

// The same, with the blocks that join few rows' dx behind them.
template <int DT, bool KC>
__global__ __launch_bounds__(256, 4) void lora_few_join_outers(WideParams p, int cb, OuterParams wide, OuterParams narrow) {
    __shared__ __attribute__((aligned(16))) char lds[outer_lds<128, 64, 1>()];
    static_assert(FEW_LDS * 4 <= outer_lds<128, 64, 1>(), "the narrow rows fit");
    const int id = (int)blockIdx.x - wide.blocks - narrow.blocks;
    if (id >= 0) few_join_block<DT, KC>(p, cb, id, reinterpret_cast<float *>(lds));
    else if ((int)blockIdx.x < wide.blocks) outer_block<DT, 128, 64, 1>(wide, blockIdx.x, lds);
    else outer_block<DT, 64, 128, 1>(narrow, (int64_t)blockIdx.x - wide.blocks, lds);
}

// ---------------------------------------------------------------------------
// Dispatch
// ---------------------------------------------------------------------------
template <class L>
LowParams low_params(const LoraLow &a) {
    LowParams q{a.rows, matrix(a.f.first), matrix(a.x), a.f.stride, a.R, a.K, (a.K + KB - 1) / KB, (a.R + L::TP - 1) / L::TP,
                (int)(((int64_t)a.rows.T + L::TQ - 1) / L::TQ), a.lists, a.splits, 0, a.partial};
    q.blocks = IsRowLow<L>::value ? a.rows.T * q.tiles_r : q.groups * q.tiles_r * q.lists * q.splits;
    return q;
}
template <class L>
hipError_t run_low(const LoraLow &a, hipStream_t stream) {
    const LowParams q = low_params<L>(a);
    hipLaunchKernelGGL(lora_low<L>, dim3((unsigned)q.blocks), dim3(L::NT), 0, stream, q);
    return hipGetLastError();
}

// f(loop type) for a factor's storage and the rank.
template <class L_>
struct Narrow {
    using L = L_;
};
template <int DT, bool KC, class F>
hipError_t with_narrow(const LoraLow &p, F &&f) {
    if (p.by_rows) return f(Narrow<RowLow<DT, KC>>());
    switch (lora_low_tile(p.R, KC)) {
    case LL_64x64: return f(Narrow<ThinLoop<DT, KC, true, 64, 64, 5>>());
    case LL_128x64: return f(Narrow<ThinLoop<DT, KC, true, 128, 64, 3>>());
    default: break;
    }
    if constexpr (KC) return f(Narrow<ThinLoop<DT, true, true, 32, 64, 6>>());
    return hipErrorInvalidValue;
}
template <int DT>
hipError_t run_lows(const LoraLow &k, const LoraLow &r, uint64_t *masks, hipStream_t stream) {
    return with_narrow<DT, true>(k, [&](auto nk) {
        return with_narrow<DT, false>(r, [&](auto nr) {
            using LK = typename decltype(nk)::L;
            using LR = typename decltype(nr)::L;
            if constexpr (LK::TP == LR::TP || (LK::TP == 32 && LR::TP == 64)) {   // what one rank and number of rows ask for
                LowParams a = low_params<LK>(k), b = low_params<LR>(r);
                if (!k.partial) a.blocks = 0;
                if (!r.partial) b.blocks = 0;
                const unsigned slabs = masks ? (unsigned)((k.rows.T + 255) / 256) : 0;
                hipLaunchKernelGGL((lora_lows<LK, LR>), dim3((unsigned)(a.blocks + b.blocks) + slabs), dim3(256), 0, stream, a, b, masks);
                return hipGetLastError();
            } else {
                return hipErrorInvalidValue;
            }
        });
    });
}

LowJoin low_join(const LoraLowJoin &a) {
    LowJoin q{a.rows, a.R, {{a.s, a.s_splits, a.s_low}, {a.ds, a.ds_splits, a.ds_low}}, 0};
    if (a.s_low || a.ds_low) q.blocks = (int)((2 * (int64_t)a.rows.T * (a.R / 4) + 255) / 256);
    return q;
}
template <class L>
WideParams wide_params(const LoraProduct &a, const LoraLowJoin &join = LoraLowJoin()) {
    return WideParams{a.rows, matrix(a.P), matrix(a.x), matrix(a.f.first), a.f.stride, a.partial, a.low_splits, a.K, a.R,
                      grid_of<L>(a.P.rows, a.x.rows, a.K, a.splits), a.whole, a.slots, a.out, a.ldo, low_join(join)};
}
template <class L>
int64_t tail_blocks(const WideParams &p) { return (int64_t)(p.g.tiles_p * p.g.tiles_q - p.whole) * (L::TP * L::TQ / 4 / 256); }

// f(loop type, stages of the adapters' slabs)
template <class L_, int DT_, int NS_>
struct Wide {
    using L = L_;
    static constexpr int DT = DT_, NS = NS_;
};
template <int DT, bool KC, class F>
hipError_t with_wide(int tile, F &&f) {
    switch (tile) {
    case LP_128x128: return f(Wide<Loop<DT, KC, true, 128, 128, 2, 2, KC ? 3 : 2, 2>, DT, 3>());
    case LP_256x256: return f(Wide<Loop<DT, KC, true, 256, 256, 2, 4, 3, 2>, DT, 3>());
    case LP_64x32: return f(Wide<ThinLoop<DT, KC, true, 64, 32, 6>, DT, 7>());
    case LP_64x64: return f(Wide<ThinLoop<DT, KC, true, 64, 64, 5>, DT, 6>());
    case LP_64x128: return f(Wide<ThinLoop<DT, KC, true, 64, 128, 3>, DT, 6>());
    default: return hipErrorInvalidValue;
    }
}
// The few rows' two launches.
unsigned few_blocks(const Grid &g, int cb) { return (unsigned)(g.tiles_p * g.tiles_q * cb); }
template <int DT, bool KC>
hipError_t join_few(const WideParams &w, int cb, hipStream_t stream) {
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((lora_few_join<DT, KC>), dim3(few_blocks(w.g, cb)), dim3(256), 0, stream, w, cb);
    return hipGetLastError();
}
template <int DT, bool KC, class L>
hipError_t run_few(const LoraProduct &a, const LoraLow &low, hipStream_t stream) {
    // the wide product's factor is stored as P is, the narrow one's the other way (an
    // input's side against an output's)
    return with_narrow<DT, KC>(low, [&](auto n) {
        using LN = typename decltype(n)::L;
        WideParams w = wide_params<L>(a);
        LowParams q = low_params<LN>(low);
        if constexpr (KC && L::TQ == 32 && LN::TP != 32) {   // up to 32 ranks, so few rows' narrow products are made row by row
            if (a.x.rows <= VEC_T) {
                w.g.splits = 1;
                const int wide = a.P.rows / 8;
                const dim3 grid((unsigned)(wide + q.blocks));
                if (a.x.rows == 1) hipLaunchKernelGGL((lora_few_vec<DT, 1, L, LN>), grid, dim3(256), 0, stream, w, q, wide);
                else if (a.x.rows == 2) hipLaunchKernelGGL((lora_few_vec<DT, 2, L, LN>), grid, dim3(256), 0, stream, w, q, wide);
                else hipLaunchKernelGGL((lora_few_vec<DT, 4, L, LN>), grid, dim3(256), 0, stream, w, q, wide);
                return join_few<DT, KC>(w, L::CB, stream);
            }
        }
        const int wide = wide_blocks(w.g, 0);
        hipLaunchKernelGGL((lora_few<L, LN>), dim3((unsigned)(wide + q.blocks)), dim3(256), 0, stream, w, q, wide);
        return join_few<DT, KC>(w, L::CB, stream);
    });
}
template <int DT, bool KC>
hipError_t few(int tile, const LoraProduct &a, const LoraLow &low, hipStream_t stream) {
    switch (tile) {
    case LP_64x32: return run_few<DT, KC, ThinLoop<DT, KC, true, 64, 32, 6>>(a, low, stream);
    case LP_64x64: return run_few<DT, KC, ThinLoop<DT, KC, true, 64, 64, 5>>(a, low, stream);
    case LP_64x128: return run_few<DT, KC, ThinLoop<DT, KC, true, 64, 128, 3>>(a, low, stream);
    default: return hipErrorInvalidValue;
    }
}
// The same where the operands' storage does not matter.
template <class F>
hipError_t with_tile(int dtype, int tile, F &&f) {
    return dtype == 0 ? with_wide<0, true>(tile, f) : with_wide<1, true>(tile, f);
}

OuterParams outer_params(const LoraOuter &a) {
    const int tp = a.narrow_p ? 64 : 128, tq = a.narrow_p ? 128 : 64;
    OuterParams q{matrix(a.P), matrix(a.Q), a.T, (a.T + 63) / 64, a.count, a.masks, (a.P.rows + tp - 1) / tp,
                  (a.Q.rows + tq - 1) / tq, a.splits, 0, a.partial, a.out_kind, a.out, a.ldo, a.stride};
    q.blocks = a.out ? a.count * q.tiles_p * q.tiles_q * a.splits : 0;
    return q;
}
template <int DT>
hipError_t join_outers(const OuterParams &w, const OuterParams &n, hipStream_t stream) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || w.splits == 1) return e;
    auto blocks = [](const OuterParams &q) { return q.out ? (int)(((int64_t)q.count * q.Q.rows * (q.P.rows / 4) + 255) / 256) : 0; };
    const int first = blocks(w);
    hipLaunchKernelGGL(lora_outer_join<DT>, dim3((unsigned)(first + blocks(n))), dim3(256), 0, stream, w, n, first);
    return hipGetLastError();
}

}  // namespace

int lora_low_tile(int R, bool kc) { return R <= 32 && kc ? LL_32x64 : R <= 64 ? LL_64x64 : LL_128x64; }
int lora_low_rows(int tile) { return tile == LL_32x64 ? 32 : tile == LL_64x64 ? 64 : 128; }

hipError_t launch_lora_low(int dtype, const LoraLow &p, hipStream_t stream) {
    if (!p.x.kc || p.by_rows) return hipErrorInvalidValue;
    auto run = [&](auto n) {
        using L = typename decltype(n)::L;
        if constexpr (IsRowLow<L>::value) return hipErrorInvalidValue;   // few rows' launch makes theirs
        else return run_low<L>(p, stream);
    };
    if (p.f.first.kc) return dtype == 0 ? with_narrow<0, true>(p, run) : with_narrow<1, true>(p, run);
    return dtype == 0 ? with_narrow<0, false>(p, run) : with_narrow<1, false>(p, run);
}
hipError_t launch_lora_lows(int dtype, const LoraLow &s, const LoraLow &ds, uint64_t *masks, hipStream_t stream) {
    const LoraLow &k = s.f.first.kc ? s : ds, &r = s.f.first.kc ? ds : s;
    if (!s.x.kc || !ds.x.kc || !k.f.first.kc || r.f.first.kc || s.R != ds.R || s.by_rows != ds.by_rows) return hipErrorInvalidValue;
    return dtype == 0 ? run_lows<0>(k, r, masks, stream) : run_lows<1>(k, r, masks, stream);
}

LossTileShape lora_tile_shape(int tile) {
    if (tile == LP_64x32) return {64, 32, 2};
    return loss_tile_shape(tile);
}
hipError_t launch_lora_product(int dtype, int tile, const LoraProduct &p, const LoraLowJoin &join, hipStream_t stream) {
    if (!p.x.kc || p.P.kc != p.f.first.kc || (p.splits > 1 && !p.slots) || (!p.partial && !p.slots)) return hipErrorInvalidValue;
    auto run = [&](auto w) {
        using W = decltype(w);
        using L = typename W::L;
        const WideParams q = wide_params<L>(p, join);
        const int joins = (q.join.blocks * 256 + L::NT - 1) / L::NT;
        hipLaunchKernelGGL((lora_product<W::DT, L, W::NS>), dim3((unsigned)(wide_blocks(q.g, q.whole) + joins)), dim3(L::NT), 0, stream, q);
        return hipGetLastError();
    };
    if (!p.P.kc) return dtype == 0 ? with_wide<0, false>(tile, run) : with_wide<1, false>(tile, run);
    return with_tile(dtype, tile, run);
}
hipError_t launch_lora_few_join(int dtype, int tile, const LoraProduct &p, const LoraLow &low, hipStream_t stream) {
    WideParams q = wide_params<ThinLoop<0, true, true, 64, 32, 6>>(p);   // every tile of few rows has 64 columns
    const int cb = lora_tile_shape(tile).q / 16;
    q.g.tiles_q = (int)((p.x.rows + 16 * cb - 1) / (16 * cb));
    q.partial = low.partial;
    q.low_splits = low.splits;
    if (p.P.kc) return dtype == 0 ? join_few<0, true>(q, cb, stream) : join_few<1, true>(q, cb, stream);
    return dtype == 0 ? join_few<0, false>(q, cb, stream) : join_few<1, false>(q, cb, stream);
}
hipError_t launch_lora_low_join(int dtype, const LoraLowJoin &p, hipStream_t stream) {
    const LowJoin q = low_join(p);
    if (!q.blocks) return hipSuccess;
    if (dtype == 0) hipLaunchKernelGGL(lora_low_join<0>, dim3((unsigned)q.blocks), dim3(256), 0, stream, q);
    else hipLaunchKernelGGL(lora_low_join<1>, dim3((unsigned)q.blocks), dim3(256), 0, stream, q);
    return hipGetLastError();
}
hipError_t launch_lora_few(int dtype, int tile, const LoraProduct &p, const LoraLow &low, hipStream_t stream) {
    if (!p.x.kc || !low.x.kc || p.P.kc != p.f.first.kc || p.P.kc != low.f.first.kc || p.R > LORA_FEW_R || p.x.rows > LORA_FEW_T)
        return hipErrorInvalidValue;
    if (p.P.kc) return dtype == 0 ? few<0, true>(tile, p, low, stream) : few<1, true>(tile, p, low, stream);
    return dtype == 0 ? few<0, false>(tile, p, low, stream) : few<1, false>(tile, p, low, stream);
}
hipError_t launch_lora_join(int dtype, int tile, const LoraProduct &p, hipStream_t stream) {
    return with_tile(dtype, tile, [&](auto w) {
        using W = decltype(w);
        const WideParams q = wide_params<typename W::L>(p);
        hipLaunchKernelGGL((lora_join<W::DT, typename W::L>), dim3((unsigned)tail_blocks<typename W::L>(q)), dim3(256), 0, stream, q);
        return hipGetLastError();
    });
}

hipError_t launch_lora_outers(int dtype, const LoraOuter &da, const LoraOuter &db, int tile, const LoraProduct *tail, const LoraLow *few,
                              hipStream_t stream) {
    const LoraOuter &w = da.narrow_p ? db : da, &n = da.narrow_p ? da : db;
    if (w.P.kc || w.Q.kc || n.P.kc || n.Q.kc || w.narrow_p || !n.narrow_p) return hipErrorInvalidValue;
    const OuterParams qw = outer_params(w), qn = outer_params(n);
    if (tail && few) {
        WideParams q = wide_params<ThinLoop<0, true, true, 64, 32, 6>>(*tail);   // every tile of few rows has 64 columns
        const int cb = lora_tile_shape(tile).q / 16;
        q.g.tiles_q = (int)((tail->x.rows + 16 * cb - 1) / (16 * cb));
        q.partial = few->partial;
        q.low_splits = few->splits;
        const dim3 grid(few_blocks(q.g, cb) + (unsigned)(qw.blocks + qn.blocks));
        auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, q, cb, qw, qn); };
        if (tail->P.kc) dtype == 0 ? run(lora_few_join_outers<0, true>) : run(lora_few_join_outers<1, true>);
        else dtype == 0 ? run(lora_few_join_outers<0, false>) : run(lora_few_join_outers<1, false>);
        return dtype == 0 ? join_outers<0>(qw, qn, stream) : join_outers<1>(qw, qn, stream);
    }
    if (!tail) {
        if (dtype == 0) hipLaunchKernelGGL(lora_outers<0>, dim3((unsigned)(qw.blocks + qn.blocks)), dim3(256), 0, stream, qw, qn);
        else hipLaunchKernelGGL(lora_outers<1>, dim3((unsigned)(qw.blocks + qn.blocks)), dim3(256), 0, stream, qw, qn);
        return dtype == 0 ? join_outers<0>(qw, qn, stream) : join_outers<1>(qw, qn, stream);
    }
    return with_tile(dtype, tile, [&](auto x) {
        using W = decltype(x);
        const WideParams q = wide_params<typename W::L>(*tail);
        const int64_t blocks = tail_blocks<typename W::L>(q) + qw.blocks + qn.blocks;
        hipLaunchKernelGGL((lora_join_outers<W::DT, typename W::L>), dim3((unsigned)blocks), dim3(256), 0, stream, q, qw, qn);
        return join_outers<W::DT>(qw, qn, stream);
    });
}

}  // namespace dgw
