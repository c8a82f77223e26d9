// tile_store.h -- what happens to a finished product tile (device code, internal to
// the library): 16-bit stores through LDS, and fp32 slots of partial sums; and the
// launches' grids (host code).
#pragma once

#include <algorithm>

#include "loss.h"
#include "tile.h"

namespace dgw {
namespace tile {

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

template <int DT>
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b) {
    if constexpr (DT == 0) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    } else {
        const f16x2 v = __builtin_bit_cast(f16x2, w);
        a = (float)v[0];
        b = (float)v[1];
    }
}
template <int DT>
__device__ __forceinline__ u32x2 pack4(f32x4 v) {
    return u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}
template <int DT>
__device__ __forceinline__ f32x4 unpack4(u32x2 w) {
    f32x4 v;
    float a, b;
    unpack2<DT>(w[0], a, b);
    v[0] = a;
    v[1] = b;
    unpack2<DT>(w[1], a, b);
    v[2] = a;
    v[3] = b;
    return v;
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

// Slot of (slice, tile): a wave's blocks one after the other, each 64 float4 (one
// a lane), so every access moves 1 KiB of contiguous memory.
template <class L>
__device__ __forceinline__ f32x4 *slot_base(float *slots, const Grid &g, int tp, int tq, int split, int wave, int lane) {
    const int64_t tile = ((int64_t)split * g.tiles_q + tq) * g.tiles_p + tp;
    return reinterpret_cast<f32x4 *>(slots + tile * (L::TP * L::TQ)) + wave * (L::RB * L::CB * 64) + lane;
}

inline Matrix matrix(const LossMatrix &m) { return Matrix{m.base, m.ld, m.rows, m.part}; }

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

inline unsigned blocks_of(const Grid &g) { return (unsigned)(g.tiles_p * g.tiles_q * g.splits); }

}  // namespace tile
}  // namespace dgw
