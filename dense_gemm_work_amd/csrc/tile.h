// tile.h -- the product tiles of the kernels of the vocabulary losses, the gated
// feed-forward block and the adapters (device code, internal to the library).
//
// One workgroup computes a TP x TQ block of sum_k P[p][k] Q[q][k] in fp32.  P is
// the dimension that lies contiguous in the result's memory (vocabulary entries
// or hidden features), Q the result's rows.  P is the matrix instruction's row
// operand, so a lane holds one row q and, in four consecutive registers, four
// consecutive p: a row's reductions (maximum, sum of exponentials) run inside a
// lane, and 16-bit results pack without any exchange between lanes.
//
// Either operand may be stored with k contiguous ([rows][k], "KC") or with its
// rows contiguous ([k][rows], "RC"), so logits, dx and dw read x, w and the
// logits' gradient as they lie and nothing is transposed in memory.  64-wide
// slabs of k move from global memory straight into LDS (16 bytes a lane, no
// registers) into NS stages; KC slabs are read with 128-bit LDS reads, RC slabs
// with the transposing 64-bit read.  The XOR swizzles leave both free of bank
// conflicts: 16 consecutive KC rows read at one chunk cover all 64 banks (their
// low three bits move the chunk), and so do the k-rows that a transposing read
// touches (four consecutive ones per 16 lanes, those of neighbouring groups 8
// apart: bits 0, 1 and 3 of k move the chunk).
//
// The products are 16x16x32 matrix instructions: on one card 4096 x 131072 x 4096
// logits took 3.13 ms on them and 3.31 ms on 32x32x16 ones, and 3.0 to 3.05 ms
// (1.44 to 1.47 PFLOP/s) since the products go back and forth along Q.  The chip
// is at its power cap there: 1.6 to 1.7 GHz with the matrix cores busy 75 % of the
// time.  Where it ran at 1.40 PFLOP/s, the same loop with every load answered by the
// L2 ran at 1.55, and on operands of zeros, which cost the least power, at 1.65.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

namespace dgw {
namespace tile {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int KB = 64;                        // k per slab: two 32-wide matrix steps
constexpr uint32_t OOB = 0x7ffffff0u;         // beyond every buffer range used here: such loads return zero
constexpr uint32_t RSRC_DW3 = 0x00020000u;    // raw buffer, 32-bit data format

__device__ __forceinline__ int swz_kc(int r) { return r & 7; }
// k-rows of 8 chunks (R = 64): two of them cover the banks, bit 0 of k says which
// half, and bits 1 and 3 move the pair of chunks that 4 lanes read.
template <int R>
__device__ __forceinline__ int swz_rc(int k) {
    if constexpr (R == 64) return (k & 2) ^ ((k >> 1) & 4);
    return ((k & 1) << 2) ^ ((k & 2) * 5) ^ ((k >> 2) & 2);
}

// D[row][col] += sum_k A[row][k] B[col][k]: lane l holds A row l % 16 and B column
// l % 16 at k = 8 (l / 16) .. + 7, and D column l % 16, rows 4 (l / 16) .. + 3.
template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ i32x4 make_rsrc(const void *base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xffff);
    r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
    r[3] = (int)RSRC_DW3;
    return r;
}

// 16 bytes a lane from global memory into 1 KiB of LDS at the wave-uniform
// `lds_addr`.  Inline assembly keeps the compiler from waiting for it before
// unrelated LDS reads (wait_vm_lgkm awaits it); the s_nop is the wait state that
// an LDS load needs after a scalar write of M0.  It writes no register.
__device__ __forceinline__ void load_lds16(i32x4 rsrc, uint32_t lds_addr, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds_addr), "v"(voff), "s"(rsrc)
                 : "memory");
}

// Wait until at most N vector-memory operations of this wave are outstanding and
// all of its LDS operations are done.
template <int N>
__device__ __forceinline__ void wait_vm_lgkm() {
    static_assert(N >= 0 && N < 64, "the counter holds 0..63");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
// The workgroup's barrier without __syncthreads()' wait for loads in flight (the
// callers wait for what they need); no memory access moves across it.
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
template <int PER>
__device__ __forceinline__ void wait_stages(int stages) {
    switch (stages) {
    case 7: wait_vm_lgkm<7 * PER <= 63 ? 7 * PER : 0>(); break;
    case 6: wait_vm_lgkm<6 * PER <= 63 ? 6 * PER : 0>(); break;
    case 5: wait_vm_lgkm<5 * PER <= 63 ? 5 * PER : 0>(); break;
    case 4: wait_vm_lgkm<4 * PER <= 63 ? 4 * PER : 0>(); break;
    case 3: wait_vm_lgkm<3 * PER>(); break;
    case 2: wait_vm_lgkm<2 * PER>(); break;
    case 1: wait_vm_lgkm<1 * PER>(); break;
    default: wait_vm_lgkm<0>(); break;
    }
}

template <int OFF>
__device__ __forceinline__ u32x4 lds_b128(uint32_t addr) {
    return *reinterpret_cast<const lds_u32x4 *>(static_cast<uintptr_t>(addr + OFF));
}
template <int OFF>
__device__ __forceinline__ u32x2 lds_tr16(uint32_t addr) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4i16 *>(static_cast<uintptr_t>(addr + OFF))));
}

// An operand of a product as it lies in memory: element (row, k) at
// base[row * ld + k] (KC) or base[k * ld + row] (RC), `rows` of them.  KC rows
// are read in chunks of 8 k, RC k-rows in chunks of 8 rows: k (KC) or rows (RC)
// rounded up to 8 must lie inside ld, and what lies there beyond k must be zero.
// A matrix may be the sum of two 16-bit parts, the second `part` elements behind
// the first; the loops that take such operands say so.
struct Matrix {
    const uint16_t *base;
    int64_t ld;
    int rows;
    int64_t part;
};

// Which rows of an operand's tile take part; the others are zeros, whatever they hold.
struct AllRows {
    __device__ __forceinline__ bool operator()(int) const { return true; }
};

// One operand's slabs: R rows by 64 k, moved by NW waves.  SRC = 2: the slabs of a
// second matrix of the same shape, ld and storage follow those of the first (the sum
// of two products in one loop: as two loops one after the other, the accumulators
// between them cost a thousand spilled registers).
template <bool KC, int R, int NW, int SRC = 1>
struct Operand {
    static constexpr int SLAB = R * KB * 2;          // bytes of one stage
    static constexpr int LOADS = R / 8 / NW;         // load instructions per wave and slab (1 KiB each)
    static_assert(LOADS >= 1 && LOADS * 8 * NW == R, "whole instructions per wave");
    static_assert(KC || R >= 64, "the swizzles of k-rows need 8 or 16 chunks");

    const char *base;
    int64_t ld;
    int K;
    uint32_t range;                // KC: bytes from base to the end of the last row
    int width;                     // RC: rows, rounded up to whole chunks
    uint32_t off[LOADS];           // the lane's byte offset at slab 0
    int kc;                        // KC: first k of the lane's chunk
    const char *base2;             // SRC = 2
    int turn;                      // its first slab

    __device__ __forceinline__ void also(const Matrix &m, int64_t row0, int slabs) {
        base2 = reinterpret_cast<const char *>(KC ? m.base + row0 * m.ld : m.base + row0);
        turn = slabs;
    }
    __device__ __forceinline__ int local(int slab) const { return SRC == 2 && slab >= turn ? slab - turn : slab; }

    template <class Keep = AllRows>
    __device__ __forceinline__ void init(const Matrix &m, int64_t row0, int K_, int wave, int lane, Keep keep = Keep()) {
        const int rows = (int)min((int64_t)R, m.rows - row0);
        ld = m.ld;
        K = K_;
        if constexpr (KC) {
            base = reinterpret_cast<const char *>(m.base + row0 * ld);
            range = (uint32_t)(((int64_t)(rows - 1) * ld + ((K + 7) & ~7)) * 2);
            width = 0;
            kc = 8 * ((lane & 7) ^ swz_kc(lane >> 3));   // the rows of one lane are a multiple of 8 apart
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                const int r = 8 * (wave * LOADS + x) + (lane >> 3);
                off[x] = r < rows && keep(r) ? (uint32_t)(r * ld + kc) * 2 : OOB;
            }
        } else {
            constexpr int CH = R / 8;                // 16-byte chunks per k-row
            base = reinterpret_cast<const char *>(m.base + row0);
            range = 0;
            width = (rows + 7) & ~7;
            kc = 0;
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                const int k = (64 / CH) * (wave * LOADS + x) + lane / CH;
                const int c = (lane % CH) ^ swz_rc<R>(k);
                off[x] = 8 * c < rows ? (uint32_t)(k * ld + 8 * c) * 2 : OOB;
            }
        }
    }

    // Buffer of slab `slab`, `shift` bytes on.
    __device__ __forceinline__ i32x4 rsrc(int slab, int64_t shift = 0) const {
        const char *base = SRC == 2 && slab >= turn ? base2 : this->base;
        const int64_t kb = (int64_t)local(slab) * KB;
        if constexpr (KC) return make_rsrc(base + shift + kb * 2, range - (uint32_t)kb * 2);
        // the range stops behind the last k-row's last chunk: width <= ld, so every
        // k-row beyond K starts outside it and reads zeros
        const int krows = (int)min((int64_t)KB, K - kb);
        return make_rsrc(base + shift + kb * ld * 2, (uint32_t)(((int64_t)(krows - 1) * ld + width) * 2));
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load(i32x4 r, int slab, int x, uint32_t dst) const {
        uint32_t o = off[x];
        if constexpr (RAGGED && KC) o = local(slab) * KB + kc < K ? o : OOB;
        load_lds16(r, dst + x * 1024, o);
    }

    // Where the lane reads its share of 16-row block `block` of the rows from
    // `first` (a multiple of 16) at matrix step `step` (32 k): one of ADDRESSES
    // registers plus a constant.  KC rows 16 apart share their swizzle, so a block
    // is a constant and a step an address; with RC it is the other way round.
    template <int BLOCKS>
    static constexpr int addresses() { return KC ? 2 : BLOCKS; }
    static constexpr int which(int block, int step) { return KC ? step : block; }
    static constexpr int constant(int block, int step) { return KC ? block * 2048 : step * 64 * R; }
    static __device__ __forceinline__ uint32_t address(uint32_t lds, int first, int lane, int number) {
        const int group = lane >> 4;
        if constexpr (KC) {
            const int r = first + (lane & 15);
            return lds + r * 128 + (((4 * number + group) ^ swz_kc(r)) << 4);
        } else {
            const int n = first + number * 16 + 4 * (lane & 3);
            const int k = 8 * group + ((lane & 15) >> 2);
            return lds + k * (2 * R) + ((((n >> 3) ^ swz_rc<R>(k)) & (R / 8 - 1)) << 4) + ((n & 7) << 1);
        }
    }
    // The fragment at `addr`: eight consecutive k of the lane's row.
    static __device__ __forceinline__ u32x4 fragment(uint32_t addr) {
        if constexpr (KC) return lds_b128<0>(addr);
        const u32x2 a = lds_tr16<0>(addr), b = lds_tr16<0>(addr + 8 * R);
        return u32x4{a[0], a[1], b[0], b[1]};
    }
};

// Work of one launch: the tiles of a TP x TQ grid, `splits` slices of k each.
struct Grid {
    int tiles_p, tiles_q;    // tiles along P and Q
    int band;                // ids run along P inside bands of this many P tiles
    int splits;              // slices of k (slowest)
    int slabs;               // slabs of k
};

// Workgroup b of n runs on XCD b % 8; each XCD gets a contiguous range of ids.
__device__ __forceinline__ int spread(int n, int b) {
    const int x = b & 7;
    return x * (n >> 3) + min(x, n & 7) + (b >> 3);
}
// Ids of tiles walk bands of `band` P tiles row by row of Q, so the tiles that run at
// once on an XCD are a compact block that shares its operands in the XCD's L2.
__device__ __forceinline__ void tile_of(const Grid &g, int id, int &tp, int &tq) {
    const int per = g.band * g.tiles_q;
    const int bnd = id / per;
    const int rows = min(g.band, g.tiles_p - bnd * g.band);
    const int w = id - bnd * per;
    tq = w / rows;
    tp = bnd * g.band + (w - tq * rows);
}
// The workgroup's tile and slice.
__device__ __forceinline__ void place(const Grid &g, int n, int b, int &tp, int &tq, int &split) {
    const int id = spread(n, b), tiles = g.tiles_p * g.tiles_q;
    split = id / tiles;
    tile_of(g, id - split * tiles, tp, tq);
}
__device__ __forceinline__ void place(const Grid &g, int &tp, int &tq, int &split) {
    place(g, (int)gridDim.x, (int)blockIdx.x, tp, tq, split);
}

// The product loop of a TP x TQ tile on WP x WQ waves with NSP stages of P and NSQ
// of Q (NSP >= NSQ).  PAIR: P's rows are TP / 2 rows each of two matrices, loaded by one
// half of the waves each into one half of a stage; a wave's blocks alternate between
// them, so a lane holds both products of a row in neighbouring blocks.
template <int DT, bool PK, bool QK, int TP_, int TQ_, int WP_, int WQ_, int NSP_, int NSQ_, bool PAIR = false, int SRC = 1>
struct Loop {
    static constexpr int TP = TP_, TQ = TQ_, WP = WP_, WQ = WQ_, NSP = NSP_, NSQ = NSQ_;
    static constexpr int NW = WP * WQ, NT = 64 * NW, WAVES = 2;   // waves resident per SIMD
    static constexpr int WAVE_P = TP / WP, WAVE_Q = TQ / WQ;
    static constexpr int RB = WAVE_P / 16, CB = WAVE_Q / 16;   // 16 x 16 blocks of a wave
    static constexpr int HB = RB / 2;                          // P blocks of half a step
    static constexpr int KINDS = PAIR ? 2 : 1;                 // matrices of P
    using OpP = Operand<PK, TP / KINDS, NW / KINDS, SRC>;
    using OpQ = Operand<QK, TQ, NW, SRC>;
    static constexpr int LOADS = OpP::LOADS + OpQ::LOADS;      // per wave and slab
    static constexpr int SLAB_P = KINDS * OpP::SLAB;
    static constexpr int QREG = NSP * SLAB_P;                  // Q's slabs lie behind P's
    static constexpr int LDS_BYTES = NSP * SLAB_P + NSQ * OpQ::SLAB;
    static constexpr int PA = OpP::template addresses<RB / KINDS>(), QA = OpQ::template addresses<CB>();
    static_assert(NSQ == 2 && (NSP == 2 || NSP == 3), "two stages, or three of P");
    static constexpr int ROUND = NSP == NSQ ? 2 : 6;           // iterations until the stages repeat

    struct Acc {
        f32x4 v[RB][CB];
    };

    int lane, wave, wp, wq;
    uint32_t lds0;
    OpP P;
    OpQ Q;
    uint32_t pa[PA], qa[QA];

    __device__ __forceinline__ Loop(char *lds) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        wp = wave % WP;
        wq = wave / WP;
        lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
#pragma unroll
        for (int i = 0; i < PA; ++i) pa[i] = OpP::address(lds0, wp * (WAVE_P / KINDS), lane, i);
#pragma unroll
        for (int i = 0; i < QA; ++i) qa[i] = OpQ::address(lds0 + QREG, wq * WAVE_Q, lane, i);
    }

    static __device__ __forceinline__ void zero(Acc &a) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) a.v[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // P's fragments of half a step, Q's of a step.
    struct FragP {
        u32x4 v[HB];
    };
    struct FragQ {
        u32x4 v[CB];
    };
    // Fragment R of what half HALF of step STEP of iteration IT (modulo ROUND)
    // needs: of the first half Q's fragments and P's, of the second P's.
    template <int IT, int STEP, int HALF, int R>
    __device__ __forceinline__ void read(FragP &p, FragQ &q) const {
        if constexpr (HALF == 0 && R > 0 && R <= CB) {
            q.v[R - 1] = OpQ::fragment(qa[OpQ::which(R - 1, STEP)] + IT % NSQ * OpQ::SLAB + OpQ::constant(R - 1, STEP));
        } else {
            constexpr int i = HALF == 0 && R > 0 ? R - CB : R, b = HALF * HB + i;
            p.v[i] = OpP::fragment(pa[OpP::which(b / KINDS, STEP)] + IT % NSP * SLAB_P + b % KINDS * OpP::SLAB +
                                   OpP::constant(b / KINDS, STEP));
        }
    }
    static constexpr int reads(int half) { return half == 0 ? HB + CB : HB; }

    // The loads of an iteration: slab sq of Q into its stage, then slab sp of P.
    struct Issue {
        i32x4 rp, rq;
        uint32_t dp, dq;
        int sp, sq;
        bool p, q;   // whether there are such slabs
    };
    __device__ __forceinline__ Issue prepare(int sp, int stp, bool p, int sq, int stq, bool q) const {
        return Issue{P.rsrc(sp), Q.rsrc(sq), lds0 + stp * SLAB_P + wave * OpP::LOADS * 1024,
                     lds0 + QREG + stq * OpQ::SLAB + wave * OpQ::LOADS * 1024, sp, sq, p, q};
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load_one(const Issue &q, int x) const {
        if (x < OpQ::LOADS) {
            if (q.q) Q.template load<RAGGED>(q.rq, q.sq, x, q.dq);
        } else if (q.p) {
            P.template load<RAGGED>(q.rp, q.sp, x - OpQ::LOADS, q.dp);
        }
    }

    // Products [M0, M1) of half HALF of a step, and evenly between them the reads of
    // the next half's fragments (half NH of step NSTEP of iteration NIT) when READ, and
    // the loads of `issue` when LOAD: the matrix pipe keeps running while they go out.
    template <int HALF, int M0, int M1, bool READ, int NIT, int NSTEP, int NH, bool LOAD, bool RAGGED>
    __device__ __forceinline__ void products(const FragP &p, const FragQ &q, Acc &acc, FragP &np, FragQ &nq,
                                             const Issue &issue) const {
        auto one = [&](auto MC) {
            constexpr int m = decltype(MC)::value, k = m - M0, n = M1 - M0;
            // back and forth along Q: one operand changes from one product to the next,
            // never both (1 % faster at the power cap)
            constexpr int hi = m / CB, j = hi & 1 ? CB - 1 - m % CB : m % CB, i = HALF * HB + hi;
            acc.v[i][j] = mfma<DT>(p.v[hi], q.v[j], acc.v[i][j]);
            constexpr int NR = READ ? reads(NH) : 0, r0 = k * NR / n, r1 = (k + 1) * NR / n;
            constexpr int NL = LOAD ? LOADS : 0, x0 = k * NL / n, x1 = (k + 1) * NL / n;
            if constexpr (r1 > r0 || x1 > x0) __builtin_amdgcn_sched_barrier(0);
            if constexpr (r1 > r0) read<NIT, NSTEP, NH, r0>(np, nq);
            if constexpr (r1 > r0 + 1) read<NIT, NSTEP, NH, r0 + 1>(np, nq);
            static_assert(r1 <= r0 + 2, "at most two reads after a product");
#pragma unroll
            for (int x = x0; x < x1; ++x) load_one<RAGGED>(issue, x);
            if constexpr (r1 > r0 || x1 > x0) __builtin_amdgcn_sched_barrier(0);
        };
        each(std::make_integer_sequence<int, M1 - M0>(), [&](auto I) { one(std::integral_constant<int, M0 + decltype(I)::value>()); });
    }
    template <class F, int... I>
    static __device__ __forceinline__ void each(std::integer_sequence<int, I...>, F &&f) {
        (f(std::integral_constant<int, I>()), ...);
    }

    // acc += the products over slabs [s0, s1) of K.  Ends with a barrier: the LDS
    // is free on return.
    template <bool RAGGED>
    __device__ __forceinline__ void run(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0, int s1,
                                        Acc &acc) {
        P.init(mp, p0, K, wave % (NW / KINDS), lane);
        Q.init(mq, q0, K, wave, lane);
        const int n = s1 - s0;
        if (n <= 0) return;
        FragP p[2];
        FragQ q[2];
        // Slabs in the order in which they are waited for: Q 0, P 0, Q 1, P 1, (P 2).
        // Iteration i then loads Q i + 2 and P i + NSP.
#pragma unroll
        for (int i = 0; i < NSP; ++i) {
            const Issue first = prepare(s0 + (i < n ? i : 0), i, i < n, s0 + (i < n ? i : 0), i % NSQ, i < NSQ && i < n);
#pragma unroll
            for (int x = 0; x < LOADS; ++x) load_one<RAGGED>(first, x);
        }
        if (n > NSP - 1) wait_vm_lgkm<LOADS + (NSP - 2) * OpP::LOADS>();
        else if (n > 1) wait_vm_lgkm<LOADS>();
        else wait_vm_lgkm<0>();
        barrier();
        each(std::make_integer_sequence<int, reads(0)>(), [&](auto R) { read<0, 0, 0, decltype(R)::value>(p[0], q[0]); });
        // Iteration i (IT modulo ROUND): four half steps, each of which reads the next
        // one's fragments while it multiplies its own.  The last hands the stages
        // over on its way: wait for this wave's loads of i + 1 (P i + 2 may still be
        // on its way) and its own reads; after the barrier every wave's loads of
        // i + 1 are there and nobody reads i's stages any more; read i + 1's first
        // fragments and load into i's stages.  STEADY: all slabs named here exist.
        auto iter = [&](int i, auto ITC, auto STEADY) {
            constexpr int it = decltype(ITC)::value, nit = (it + 1) % ROUND, NM = HB * CB, BAR = NM / 4;
            constexpr bool steady = decltype(STEADY)::value;
            const Issue none{};
            __builtin_amdgcn_sched_barrier(0);
            products<0, 0, NM, true, it, 0, 1, false, RAGGED>(p[0], q[0], acc, p[1], q[1], none);
            products<1, 0, NM, true, it, 1, 0, false, RAGGED>(p[1], q[0], acc, p[0], q[1], none);
            products<0, 0, NM, true, it, 1, 1, false, RAGGED>(p[0], q[1], acc, p[1], q[0], none);
            products<1, 0, BAR, false, it, 0, 0, false, RAGGED>(p[1], q[1], acc, p[0], q[0], none);
            if (steady || i + 1 < n) {
                __builtin_amdgcn_sched_barrier(0);
                if (NSP > 2 && (steady || i + 2 < n)) wait_vm_lgkm<(NSP - 2) * OpP::LOADS>();
                else wait_vm_lgkm<0>();
                barrier();
                __builtin_amdgcn_sched_barrier(0);
                const bool more_p = steady || i + NSP < n, more_q = steady || i + NSQ < n;
                products<1, BAR, NM, true, nit, 0, 0, true, RAGGED>(
                    p[1], q[1], acc, p[0], q[0],
                    prepare(s0 + (more_p ? i + NSP : i), it % NSP, more_p, s0 + (more_q ? i + NSQ : i), it % NSQ, more_q));
            } else {
                products<1, BAR, NM, false, it, 0, 0, false, RAGGED>(p[1], q[1], acc, p[0], q[0], none);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        int i = 0;
        for (; i + ROUND + NSP <= n; i += ROUND)
            each(std::make_integer_sequence<int, ROUND>(), [&](auto I) { iter(i + decltype(I)::value, I, std::true_type()); });
        for (; i < n; i += ROUND)
            each(std::make_integer_sequence<int, ROUND>(), [&](auto I) {
                if (i + decltype(I)::value < n) iter(i + decltype(I)::value, I, std::false_type());
            });
        wait_vm_lgkm<0>();
        barrier();
    }
    __device__ __forceinline__ void run_any(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0, int s1,
                                            Acc &acc) {
        if (K % KB == 0) run<false>(mp, p0, mq, q0, K, s0, s1, acc);
        else run<true>(mp, p0, mq, q0, K, s0, s1, acc);
    }
    // SRC = 2, before run: the second product, over the same K (its slabs count on).
    __device__ __forceinline__ void also(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K) {
        P.also(mp, p0, (K + KB - 1) / KB);
        Q.also(mq, q0, (K + KB - 1) / KB);
    }
    // PAIR: the one of P's matrices that this wave loads.
    __device__ __forceinline__ const Matrix &pick(const Matrix &first, const Matrix &second) const {
        return wave < NW / 2 ? first : second;
    }

    __device__ __forceinline__ bool active() const { return true; }

    // Register e of block (i, j) is element (p, q) of the tile (PAIR: blocks 2 i and
    // 2 i + 1 are element p_of(i, e) of either matrix).
    __device__ __forceinline__ int p_of(int i, int e) const { return wp * (WAVE_P / KINDS) + i * 16 + 4 * (lane >> 4) + e; }
    __device__ __forceinline__ int q_of(int j) const { return wq * WAVE_Q + j * 16 + (lane & 15); }
};

// The product loop for few rows of Q, where P's stream from memory is the cost.
// Four waves: wave 2 h + s takes half h of P's rows and matrix step s of every
// slab, so every staged byte of P is read from LDS once, and a chain of fp32
// additions is half as long.  Small tiles and several stages keep enough bytes in
// flight per CU.  After the loop the two waves of a half swap sums through LDS:
// each then owns half of their blocks (of a 32-row tile, which has one block a
// half, the wave of step 0 owns it and the other nothing), and the members below
// describe that state, as Loop's do.  PARTS = 2: Q is the sum of two parts, both
// staged and multiplied with the same fragments of P.  PAIR: P's halves are TP / 2 rows
// each of two matrices.
template <int DT, bool PK, bool QK, int TP_, int TQ_, int NS_, int PARTS = 1, bool PAIR = false, int SRC = 1>
struct ThinLoop {
    static constexpr int TP = TP_, TQ = TQ_, NS = NS_;
    static constexpr int NW = 4, NT = 256;
    static constexpr int PB = TP / 32;                         // P blocks of a wave during the loop
    static constexpr int RB = PB > 1 ? PB / 2 : 1, CB = TQ / 16;
    static constexpr int WAVE_P = 16 * RB, WAVE_Q = TQ, WP = TP / WAVE_P, WQ = 1;
    static constexpr int KINDS = PAIR ? 2 : 1;                 // matrices of P
    using OpP = Operand<PK, TP / KINDS, NW / KINDS, SRC>;
    using OpQ = Operand<QK, TQ, NW, SRC>;
    static constexpr int LOADS = OpP::LOADS + PARTS * OpQ::LOADS;
    static constexpr int SLAB_P = KINDS * OpP::SLAB, STAGE = SLAB_P + PARTS * OpQ::SLAB;
    static constexpr int LDS_BYTES = NS * STAGE, WAVES = 2 * LDS_BYTES <= 160 * 1024 ? 2 : 1;
    static constexpr int PA = PK ? 1 : PB, QA = QK ? 1 : CB;
    static_assert(PB == 1 || PB == 2 || PB == 4, "32, 64 or 128 rows of P");
    static_assert(NS >= 2 && NS <= 8 && (NS - 1) * LOADS < 64, "the wait counter holds the loads in flight");
    static_assert(NW * RB * CB * 1024 <= LDS_BYTES, "the sums that are swapped fit");

    struct Acc {
        f32x4 v[RB][CB];
    };

    int lane, wave, wp, wq;
    uint32_t lds0;
    char *lds_;
    OpP P;
    OpQ Q;
    int64_t qpart;   // bytes from Q's first part to its second
    uint32_t pa[PA], qa[QA];

    __device__ __forceinline__ ThinLoop(char *lds) : lds_(lds) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        wp = PB > 1 ? wave : wave >> 1;
        wq = 0;
        const int step = wave & 1;
        lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
#pragma unroll
        for (int i = 0; i < PA; ++i)
            pa[i] = OpP::address(PAIR ? lds0 + (wave >> 1) * OpP::SLAB : lds0, PAIR ? 0 : (wave >> 1) * (TP / 2), lane,
                                 PK ? step : i) + (PK ? 0 : OpP::constant(0, step));
#pragma unroll
        for (int i = 0; i < QA; ++i)
            qa[i] = OpQ::address(lds0 + SLAB_P, 0, lane, QK ? step : i) + (QK ? 0 : OpQ::constant(0, step));
    }

    static __device__ __forceinline__ void zero(Acc &a) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) a.v[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    struct Frags {
        u32x4 p[PB], q[PARTS][CB];
    };
    __device__ __forceinline__ void read(Frags &f, int st) const {
        const uint32_t o = st * STAGE;
#pragma unroll
        for (int i = 0; i < PB; ++i) f.p[i] = OpP::fragment(pa[PK ? 0 : i] + o + (PK ? OpP::constant(i, 0) : 0));
#pragma unroll
        for (int x = 0; x < PARTS; ++x)
#pragma unroll
            for (int j = 0; j < CB; ++j)
                f.q[x][j] = OpQ::fragment(qa[QK ? 0 : j] + o + x * OpQ::SLAB + (QK ? OpQ::constant(j, 0) : 0));
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load_all(int slab, int st) const {
        const i32x4 rp = P.rsrc(slab);
        const uint32_t dp = lds0 + st * STAGE + wave * OpP::LOADS * 1024;
        const uint32_t dq = lds0 + st * STAGE + SLAB_P + wave * OpQ::LOADS * 1024;
#pragma unroll
        for (int x = 0; x < OpP::LOADS; ++x) P.template load<RAGGED>(rp, slab, x, dp);
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
            const i32x4 rq = Q.rsrc(slab, part * qpart);
#pragma unroll
            for (int x = 0; x < OpQ::LOADS; ++x) Q.template load<RAGGED>(rq, slab, x, dq + part * OpQ::SLAB);
        }
    }

    template <bool RAGGED, class Keep = AllRows>
    __device__ __forceinline__ void run(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0, int s1,
                                        Acc &out, Keep keep = Keep()) {
        P.init(mp, p0, K, wave % (NW / KINDS), lane);
        Q.init(mq, q0, K, wave, lane, keep);
        qpart = 2 * mq.part;
        const int n = s1 - s0;
        if (n <= 0) return;
        f32x4 acc[PB][CB];
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = 0; i < min(NS, n); ++i) load_all<RAGGED>(s0 + i, i);
        wait_stages<LOADS>(min(NS, n) - 1);
        barrier();
        Frags f[2];
        read(f[0], 0);
        int st = 0;   // stage of iteration i
        // Iteration i: this wave's loads of i + 1 and its reads of i are done; after
        // the barrier every wave's are, so slab i + NS may go into stage i; read
        // i + 1, multiply i.
        auto iter = [&](int i, Frags &cur, Frags &next) {
            __builtin_amdgcn_sched_barrier(0);
            wait_stages<LOADS>(max(0, min(NS - 2, n - i - 2)));
            barrier();
            __builtin_amdgcn_sched_barrier(0);
            if (i + NS < n) load_all<RAGGED>(s0 + i + NS, st);
            st = st + 1 == NS ? 0 : st + 1;
            if (i + 1 < n) read(next, st);
#pragma unroll
            for (int a = 0; a < PB; ++a)
#pragma unroll
                for (int b = 0; b < CB; ++b)
#pragma unroll
                    for (int x = PARTS - 1; x >= 0; --x) acc[a][b] = mfma<DT>(cur.p[a], cur.q[x][b], acc[a][b]);
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int i = 0; i < n; i += 2) {
            iter(i, f[0], f[1]);
            if (i + 1 < n) iter(i + 1, f[1], f[0]);
        }
        wait_vm_lgkm<0>();
        barrier();
        // a wave's gift to its partner, [wave][block][lane]
        f32x4 *buf = reinterpret_cast<f32x4 *>(lds_);
        const bool second = (threadIdx.x >> 6) & 1;
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                // by value: chosen by address the sums would go through memory
                const f32x4 low = acc[i][j], high = acc[PB > 1 ? RB + i : i][j];
                f32x4 give;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    give[e] = second ? low[e] : high[e];
                    out.v[i][j][e] = second ? high[e] : low[e];
                }
                buf[(wave * RB * CB + i * CB + j) * 64 + lane] = give;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) out.v[i][j] += buf[((wave ^ 1) * RB * CB + i * CB + j) * 64 + lane];
        __syncthreads();
    }
    template <class Keep = AllRows>
    __device__ __forceinline__ void run_any(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0,
                                            int s1, Acc &acc, Keep keep = Keep()) {
        if (K % KB == 0) run<false>(mp, p0, mq, q0, K, s0, s1, acc, keep);
        else run<true>(mp, p0, mq, q0, K, s0, s1, acc, keep);
    }
    __device__ __forceinline__ void also(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K) {
        P.also(mp, p0, (K + KB - 1) / KB);
        Q.also(mq, q0, (K + KB - 1) / KB);
    }
    __device__ __forceinline__ const Matrix &pick(const Matrix &first, const Matrix &second) const {
        return wave < NW / 2 ? first : second;
    }

    __device__ __forceinline__ bool active() const { return PB > 1 || !(wave & 1); }
    __device__ __forceinline__ int p_of(int i, int e) const { return wp * WAVE_P + i * 16 + 4 * (lane >> 4) + e; }
    __device__ __forceinline__ int q_of(int j) const { return j * 16 + (lane & 15); }
};

}  // namespace tile
}  // namespace dgw
