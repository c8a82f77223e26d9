// tile.h -- the product tiles of the vocabulary-loss kernels (device code,
// internal to the library).
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
// conflicts (16 consecutive KC rows cover all 64 banks; the four k-rows that a
// transposing read touches fall on distinct ones).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

namespace dgw {
namespace tile {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

constexpr int KB = 64;                        // k per slab: four 16-wide matrix steps
constexpr uint32_t OOB = 0x7ffffff0u;         // beyond every buffer range used here: such loads return zero
constexpr uint32_t RSRC_DW3 = 0x00020000u;    // raw buffer, 32-bit data format

__device__ __forceinline__ int swz_kc(int r) { return (r & 7) ^ ((r >> 3) & 3); }
__device__ __forceinline__ int swz_rc(int k) { return ((k & 1) << 2) ^ ((k & 2) * 5); }

template <int DT>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (DT == 0)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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
struct Matrix {
    const uint16_t *base;
    int64_t ld;
    int rows;
};

// One operand's slabs: R rows by 64 k, moved by NW waves.
template <bool KC, int R, int NW>
struct Operand {
    static constexpr int SLAB = R * KB * 2;          // bytes of one stage
    static constexpr int LOADS = R / 8 / NW;         // load instructions per wave and slab (1 KiB each)
    static_assert(LOADS >= 1 && LOADS * 8 * NW == R, "whole instructions per wave");
    static_assert(KC || R >= 128, "the swizzle of k-rows needs 16 chunks");

    const char *base;
    int64_t ld;
    int K;
    uint32_t range;                // KC: bytes from base to the end of the last row
    int width;                     // RC: rows, rounded up to whole chunks
    uint32_t off[LOADS];           // the lane's byte offset at slab 0
    int kc[LOADS];                 // KC: first k of the lane's chunk

    __device__ __forceinline__ void init(const Matrix &m, int64_t row0, int K_, int wave, int lane) {
        const int rows = (int)min((int64_t)R, m.rows - row0);
        ld = m.ld;
        K = K_;
        if constexpr (KC) {
            base = reinterpret_cast<const char *>(m.base + row0 * ld);
            range = (uint32_t)(((int64_t)(rows - 1) * ld + ((K + 7) & ~7)) * 2);
            width = 0;
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                const int r = 8 * (wave * LOADS + x) + (lane >> 3);
                const int c = (lane & 7) ^ swz_kc(r);
                off[x] = r < rows ? (uint32_t)(r * ld + 8 * c) * 2 : OOB;
                kc[x] = 8 * c;
            }
        } else {
            constexpr int CH = R / 8;                // 16-byte chunks per k-row
            base = reinterpret_cast<const char *>(m.base + row0);
            range = 0;
            width = (rows + 7) & ~7;
#pragma unroll
            for (int x = 0; x < LOADS; ++x) {
                const int k = (64 / CH) * (wave * LOADS + x) + lane / CH;
                const int c = (lane % CH) ^ swz_rc(k);
                off[x] = 8 * c < rows ? (uint32_t)(k * ld + 8 * c) * 2 : OOB;
                kc[x] = k;
            }
        }
    }

    // Buffer of slab `slab`.
    __device__ __forceinline__ i32x4 rsrc(int slab) const {
        const int64_t kb = (int64_t)slab * KB;
        if constexpr (KC) return make_rsrc(base + kb * 2, range - (uint32_t)kb * 2);
        // the range stops behind the last k-row's last chunk: width <= ld, so every
        // k-row beyond K starts outside it and reads zeros
        const int krows = (int)min((int64_t)KB, K - kb);
        return make_rsrc(base + kb * ld * 2, (uint32_t)(((int64_t)(krows - 1) * ld + width) * 2));
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load(i32x4 r, int slab, int x, uint32_t dst) const {
        uint32_t o = off[x];
        if constexpr (RAGGED) o = slab * KB + kc[x] < K ? o : OOB;
        load_lds16(r, dst + x * 1024, o);
    }

    // Where the lane reads 32-row block 0 of the wave's rows (from `first`, a
    // multiple of 32) at k-step 0.
    static __device__ __forceinline__ uint32_t read_base(uint32_t lds, int first, int lane, int kk, int block) {
        const int half = lane >> 5;
        if constexpr (KC) {
            const int r = lane & 31;
            return lds + first * 128 + r * 128 + ((((2 * kk + half) ^ swz_kc(r)) & 7) << 4);
        } else {
            const int n = first + block * 32 + ((lane >> 4) & 1) * 16 + 4 * (lane & 3);
            const int k = 8 * half + ((lane & 15) >> 2);
            return lds + k * (2 * R) + ((((n >> 3) ^ swz_rc(k)) & (R / 8 - 1)) << 4) + ((n & 7) << 1);
        }
    }
};

// Work of one launch: the tiles of a TP x TQ grid, `splits` slices of k each.
struct Grid {
    int tiles_p, tiles_q;    // tiles along P and Q
    int band;                // ids run along P inside bands of this many P tiles
    int splits;              // slices of k (slowest)
    int slabs;               // 64-wide slabs of k
};

// The workgroup's tile and slice.  Workgroup b runs on XCD b % 8; each XCD gets a
// contiguous range of ids, and ids walk bands of `band` P tiles row by row of Q,
// so the tiles that run at once on an XCD are a compact block that shares its
// operands in the XCD's L2.
__device__ __forceinline__ void place(const Grid &g, int &tp, int &tq, int &split) {
    const int n = (int)gridDim.x, b = (int)blockIdx.x, x = b & 7;
    int id = x * (n >> 3) + min(x, n & 7) + (b >> 3);
    const int tiles = g.tiles_p * g.tiles_q;
    split = id / tiles;
    id -= split * tiles;
    const int per = g.band * g.tiles_q;
    const int bnd = id / per;
    const int rows = min(g.band, g.tiles_p - bnd * g.band);
    const int w = id - bnd * per;
    tq = w / rows;
    tp = bnd * g.band + (w - tq * rows);
}

// The product loop of a TP x TQ tile on WP x WQ waves with NS stages.
template <int DT, bool PK, bool QK, int TP_, int TQ_, int WP_, int WQ_, int NS_>
struct Loop {
    static constexpr int TP = TP_, TQ = TQ_, WP = WP_, WQ = WQ_, NS = NS_;
    static constexpr int NW = WP * WQ, NT = 64 * NW;
    static constexpr int WAVE_P = TP / WP, WAVE_Q = TQ / WQ;
    static constexpr int RB = WAVE_P / 32, CB = WAVE_Q / 32;   // 32 x 32 blocks of a wave
    using OpP = Operand<PK, TP, NW>;
    using OpQ = Operand<QK, TQ, NW>;
    static constexpr int LOADS = OpP::LOADS + OpQ::LOADS;      // per wave and slab
    static constexpr int QREG = NS * OpP::SLAB;                // Q's slabs lie behind P's
    static constexpr int LDS_BYTES = NS * (OpP::SLAB + OpQ::SLAB);
    static_assert(NS >= 2 && NS <= 4, "two to four stages");

    struct Acc {
        f32x16 v[RB][CB];
    };
    struct Frags {
        u32x4 p[RB], q[CB];
    };

    int lane, wave, wp, wq;
    uint32_t lds0;
    OpP P;
    OpQ Q;
    uint32_t pa[PK ? 4 : RB], qa[QK ? 4 : CB];

    __device__ __forceinline__ Loop(char *lds) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        wp = wave % WP;
        wq = wave / WP;
        lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
#pragma unroll
        for (int i = 0; i < (PK ? 4 : RB); ++i) pa[i] = OpP::read_base(lds0, wp * WAVE_P, lane, PK ? i : 0, PK ? 0 : i);
#pragma unroll
        for (int i = 0; i < (QK ? 4 : CB); ++i)
            qa[i] = OpQ::read_base(lds0 + QREG, wq * WAVE_Q, lane, QK ? i : 0, QK ? 0 : i);
    }

    static __device__ __forceinline__ void zero(Acc &a) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) a.v[i][j][e] = 0.0f;
    }

    template <int ST, int KK>
    __device__ __forceinline__ void read(Frags &f) const {
        if constexpr (PK) {
#pragma unroll
            for (int i = 0; i < RB; ++i) f.p[i] = lds_b128<ST * OpP::SLAB>(pa[KK] + i * 4096);
        } else {
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const u32x2 a = lds_tr16<ST * OpP::SLAB + KK * 32 * TP>(pa[i]);
                const u32x2 b = lds_tr16<ST * OpP::SLAB + KK * 32 * TP + 8 * TP>(pa[i]);
                f.p[i] = u32x4{a[0], a[1], b[0], b[1]};
            }
        }
        if constexpr (QK) {
#pragma unroll
            for (int j = 0; j < CB; ++j) f.q[j] = lds_b128<ST * OpQ::SLAB>(qa[KK] + j * 4096);
        } else {
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                const u32x2 a = lds_tr16<ST * OpQ::SLAB + KK * 32 * TQ>(qa[j]);
                const u32x2 b = lds_tr16<ST * OpQ::SLAB + KK * 32 * TQ + 8 * TQ>(qa[j]);
                f.q[j] = u32x4{a[0], a[1], b[0], b[1]};
            }
        }
    }

    static __device__ __forceinline__ void mma(const Frags &f, Acc &acc) {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) acc.v[i][j] = mfma<DT>(f.p[i], f.q[j], acc.v[i][j]);
    }

    // The loads of one slab into one stage.
    struct Issue {
        i32x4 rp, rq;
        uint32_t dp, dq;
        int slab;
    };
    __device__ __forceinline__ Issue prepare(int slab, int st) const {
        return Issue{P.rsrc(slab), Q.rsrc(slab), lds0 + st * OpP::SLAB + wave * OpP::LOADS * 1024,
                     lds0 + QREG + st * OpQ::SLAB + wave * OpQ::LOADS * 1024, slab};
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load_one(const Issue &q, int x) const {
        if (x < OpP::LOADS) P.template load<RAGGED>(q.rp, q.slab, x, q.dp);
        else Q.template load<RAGGED>(q.rq, q.slab, x - OpP::LOADS, q.dq);
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load_all(int slab, int st) const {
        const Issue q = prepare(slab, st);
#pragma unroll
        for (int x = 0; x < LOADS; ++x) load_one<RAGGED>(q, x);
    }
    // f's products with the loads of `q` (when `load`) between them, so that the
    // matrix pipe keeps running while they go out
    template <bool RAGGED>
    __device__ __forceinline__ void mma_load(const Frags &f, Acc &acc, bool load, const Issue &q) const {
        constexpr int NM = RB * CB;
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                acc.v[i][j] = mfma<DT>(f.p[i], f.q[j], acc.v[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (load) {
                    const int m = i * CB + j;
#pragma unroll
                    for (int x = m * LOADS / NM; x < (m + 1) * LOADS / NM; ++x) load_one<RAGGED>(q, x);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
    }

    // acc += the products over slabs [s0, s1) of K.  Ends with a barrier: the LDS
    // is free on return.
    template <bool RAGGED>
    __device__ __forceinline__ void run(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0, int s1,
                                        Acc &acc) {
        P.init(mp, p0, K, wave, lane);
        Q.init(mq, q0, K, wave, lane);
        const int n = s1 - s0;
        if (n <= 0) return;
        Frags f[2];
        load_all<RAGGED>(s0, 0);
        if (n > 1) load_all<RAGGED>(s0 + 1, 1);
        if (NS > 2 && n > 2) load_all<RAGGED>(s0 + 2, 2 % NS);
        if (NS > 3 && n > 3) load_all<RAGGED>(s0 + 3, 3 % NS);
        wait_stages<LOADS>(min(NS, n) - 1);
        __builtin_amdgcn_s_barrier();
        read<0, 0>(f[0]);
        // Iteration i on stage ST: k-steps 0..2 read the next step's fragments and
        // multiply the current ones.  Step 3 hands the stage over: wait for this
        // wave's loads of i + 1 and its reads of (i, 3); after the barrier every
        // wave's loads of i + 1 are there and nobody reads stage ST any more; read
        // (i + 1, 0), then multiply step 3 while slab i + NS goes into stage ST.
        auto iter = [&](int i, auto STC) {
            constexpr int st = decltype(STC)::value;
            __builtin_amdgcn_sched_barrier(0);
            read<st, 1>(f[1]);
            mma(f[0], acc);
            __builtin_amdgcn_sched_barrier(0);
            read<st, 2>(f[0]);
            mma(f[1], acc);
            __builtin_amdgcn_sched_barrier(0);
            read<st, 3>(f[1]);
            mma(f[0], acc);
            __builtin_amdgcn_sched_barrier(0);
            if (i + 1 < n) {
                wait_stages<LOADS>(max(0, min(NS - 2, n - i - 2)));
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                read<(st + 1) % NS, 0>(f[0]);
            }
            const bool more = i + NS < n;
            mma_load<RAGGED>(f[1], acc, more, prepare(s0 + (more ? i + NS : i), st));
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int i = 0; i < n; i += NS) {
            iter(i, std::integral_constant<int, 0>());
            if (i + 1 < n) iter(i + 1, std::integral_constant<int, 1>());
            if constexpr (NS > 2)
                if (i + 2 < n) iter(i + 2, std::integral_constant<int, 2>());
            if constexpr (NS > 3)
                if (i + 3 < n) iter(i + 3, std::integral_constant<int, 3>());
        }
        wait_vm_lgkm<0>();
        __builtin_amdgcn_s_barrier();
    }
    __device__ __forceinline__ void run_any(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0,
                                            int s1, Acc &acc) {
        if (K % KB == 0) run<false>(mp, p0, mq, q0, K, s0, s1, acc);
        else run<true>(mp, p0, mq, q0, K, s0, s1, acc);
    }

    __device__ __forceinline__ bool active() const { return true; }

    // Register e of block (i, j) is element (p, q) of the tile.
    __device__ __forceinline__ int p_of(int i, int e) const {
        return wp * WAVE_P + i * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
    }
    __device__ __forceinline__ int q_of(int j) const { return wq * WAVE_Q + j * 32 + (lane & 31); }
};

// The product loop for few rows of Q, where P's stream from memory is the cost:
// four waves that split every slab's four k-steps between them, each holding the
// whole TP x TQ tile's sums over a quarter of k.  So every staged byte is read
// from LDS once (P) or once per P block (Q), and a chain of fp32 additions is a
// quarter as long.  Small tiles and several stages keep enough bytes in flight
// per CU.  After the loop the waves add their sums through LDS in wave order:
// wave w < TP / 32 then owns 32-row block w (the others own nothing), and the
// members below describe that state, as Loop's do.
template <int DT, bool PK, bool QK, int TP_, int TQ_, int NS_>
struct ThinLoop {
    static constexpr int TP = TP_, TQ = TQ_, NS = NS_;
    static constexpr int NW = 4, NT = 256;
    static constexpr int WP = TP / 32, WQ = 1;
    static constexpr int WAVE_P = 32, WAVE_Q = TQ;
    static constexpr int RB = 1, CB = TQ / 32;
    static constexpr int PB = TP / 32;                         // P blocks during the loop
    using OpP = Operand<PK, TP, NW>;
    using OpQ = Operand<QK, TQ, NW>;
    static constexpr int LOADS = OpP::LOADS + OpQ::LOADS;
    static constexpr int STAGE = OpP::SLAB + OpQ::SLAB;
    static constexpr int MERGE_BYTES = 4 * PB * 4096;          // four waves' sums of one block column
    static constexpr int LDS_BYTES = NS * STAGE > MERGE_BYTES ? NS * STAGE : MERGE_BYTES;
    static_assert(NS >= 2 && NS <= 8 && (NS - 1) * LOADS < 64, "the wait counter holds the loads in flight");
    static_assert(PB <= 4, "a wave per block");

    struct Acc {
        f32x16 v[RB][CB];
    };

    int lane, wave, wp, wq;
    uint32_t lds0;
    char *lds_;
    OpP P;
    OpQ Q;
    uint32_t pa[PK ? 1 : PB], qa[QK ? 1 : CB];

    __device__ __forceinline__ ThinLoop(char *lds) : lds_(lds) {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        wp = wave;
        wq = 0;
        lds0 = (uint32_t)reinterpret_cast<uintptr_t>((const lds_void *)lds);
        // the wave's k-step: a chunk of KC rows, 16 k-rows of RC slabs
#pragma unroll
        for (int i = 0; i < (PK ? 1 : PB); ++i)
            pa[i] = OpP::read_base(lds0, 0, lane, wave, i) + (PK ? 0 : wave * 32 * TP);
#pragma unroll
        for (int i = 0; i < (QK ? 1 : CB); ++i)
            qa[i] = OpQ::read_base(lds0 + OpP::SLAB, 0, lane, wave, i) + (QK ? 0 : wave * 32 * TQ);
    }

    static __device__ __forceinline__ void zero(Acc &a) {
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) a.v[0][j][e] = 0.0f;
    }

    struct Frags {
        u32x4 p[PB], q[CB];
    };
    __device__ __forceinline__ void read(Frags &f, int st) const {
        const uint32_t o = st * STAGE;
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            if constexpr (PK) {
                f.p[i] = lds_b128<0>(pa[0] + o + i * 4096);
            } else {
                const u32x2 a = lds_tr16<0>(pa[i] + o), b = lds_tr16<8 * TP>(pa[i] + o);
                f.p[i] = u32x4{a[0], a[1], b[0], b[1]};
            }
        }
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            if constexpr (QK) {
                f.q[j] = lds_b128<0>(qa[0] + o + j * 4096);
            } else {
                const u32x2 a = lds_tr16<0>(qa[j] + o), b = lds_tr16<8 * TQ>(qa[j] + o);
                f.q[j] = u32x4{a[0], a[1], b[0], b[1]};
            }
        }
    }
    template <bool RAGGED>
    __device__ __forceinline__ void load_all(int slab, int st) const {
        const i32x4 rp = P.rsrc(slab), rq = Q.rsrc(slab);
        const uint32_t dp = lds0 + st * STAGE + wave * OpP::LOADS * 1024;
        const uint32_t dq = lds0 + st * STAGE + OpP::SLAB + wave * OpQ::LOADS * 1024;
#pragma unroll
        for (int x = 0; x < OpP::LOADS; ++x) P.template load<RAGGED>(rp, slab, x, dp);
#pragma unroll
        for (int x = 0; x < OpQ::LOADS; ++x) Q.template load<RAGGED>(rq, slab, x, dq);
    }

    template <bool RAGGED>
    __device__ __forceinline__ void run(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0, int s1,
                                        Acc &out) {
        P.init(mp, p0, K, wave, lane);
        Q.init(mq, q0, K, wave, lane);
        const int n = s1 - s0;
        if (n <= 0) return;
        f32x16 acc[PB][CB];
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
        for (int i = 0; i < min(NS, n); ++i) load_all<RAGGED>(s0 + i, i);
        wait_stages<LOADS>(min(NS, n) - 1);
        __builtin_amdgcn_s_barrier();
        Frags f[2];
        read(f[0], 0);
        int st = 0;   // stage of iteration i
        // Iteration i: this wave's loads of i + 1 and its reads of i are done; after
        // the barrier every wave's are, so slab i + NS may go into stage i; read
        // i + 1, multiply i.
        auto iter = [&](int i, Frags &cur, Frags &next) {
            __builtin_amdgcn_sched_barrier(0);
            wait_stages<LOADS>(max(0, min(NS - 2, n - i - 2)));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            if (i + NS < n) load_all<RAGGED>(s0 + i + NS, st);
            st = st + 1 == NS ? 0 : st + 1;
            if (i + 1 < n) read(next, st);
#pragma unroll
            for (int a = 0; a < PB; ++a)
#pragma unroll
                for (int b = 0; b < CB; ++b) acc[a][b] = mfma<DT>(cur.p[a], cur.q[b], acc[a][b]);
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int i = 0; i < n; i += 2) {
            iter(i, f[0], f[1]);
            if (i + 1 < n) iter(i + 1, f[1], f[0]);
        }
        wait_vm_lgkm<0>();
        __builtin_amdgcn_s_barrier();
        // the waves' sums of one block column at a time, [wave][block][quad][lane]
        f32x4 *buf = reinterpret_cast<f32x4 *>(lds_);
#pragma unroll
        for (int j = 0; j < CB; ++j) {
#pragma unroll
            for (int i = 0; i < PB; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    buf[(wave * PB + i) * 256 + g * 64 + lane] =
                        f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            __syncthreads();
            if (active()) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    f32x4 v = buf[wave * 256 + g * 64 + lane];
#pragma unroll
                    for (int w = 1; w < 4; ++w) v += buf[(w * PB + wave) * 256 + g * 64 + lane];
#pragma unroll
                    for (int x = 0; x < 4; ++x) out.v[0][j][4 * g + x] = v[x];
                }
            }
            __syncthreads();
        }
    }
    __device__ __forceinline__ void run_any(const Matrix &mp, int64_t p0, const Matrix &mq, int64_t q0, int K, int s0,
                                            int s1, Acc &acc) {
        if (K % KB == 0) run<false>(mp, p0, mq, q0, K, s0, s1, acc);
        else run<true>(mp, p0, mq, q0, K, s0, s1, acc);
    }

    __device__ __forceinline__ bool active() const { return wave < WP; }
    __device__ __forceinline__ int p_of(int, int e) const { return wp * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3); }
    __device__ __forceinline__ int q_of(int j) const { return j * 32 + (lane & 31); }
};

}  // namespace tile
}  // namespace dgw
