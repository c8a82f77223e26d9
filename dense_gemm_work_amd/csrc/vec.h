// vec.h -- products of at most four rows with weights whose k is contiguous (device
// code, internal to the library).
//
// With so few rows the weights' stream is all there is, and what a tile's stages,
// slices and joins cost is latency.  Four waves share a few rows of the weights, a
// quarter of k each: 16 bytes a lane straight into registers, fp32 multiply-adds, one
// reduction at the end.  Every load of a workgroup is in flight at once, and the
// result needs no launch that joins slices.  (One token, 1536 x 4096: gate and up 8.3 us on 32 x 32
// tiles.)
#pragma once

#include "tile_store.h"

namespace dgw {
namespace tile {

constexpr int VEC_T = 4;   // most rows

struct f32x8 {
    float v[8];
};
template <int DT>
__device__ __forceinline__ f32x8 unpack8(u32x4 w) {
    f32x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<DT>(w[i], r.v[2 * i], r.v[2 * i + 1]);
    return r;
}

// Eight values of row t of an operand of 16-bit or fp32 values at k.
template <int DT>
struct Rows16 {
    const uint16_t *base;
    int64_t ld;
    __device__ __forceinline__ f32x8 operator()(int t, int k) const {
        return unpack8<DT>(*reinterpret_cast<const u32x4 *>(base + t * ld + k));
    }
};
struct Rows32 {
    const float *base;
    int64_t ld;
    __device__ __forceinline__ f32x8 operator()(int t, int k) const {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(base + t * ld + k), b = *reinterpret_cast<const f32x4 *>(base + t * ld + k + 4);
        return f32x8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
};

// red[wave][row i][t] = the wave's share of sum_k w_i[k] x(t, k), for N rows of weights and
// T <= VEC_T rows of x, of which those from `rows` on are left out.  256 threads; ends
// with a barrier.
template <int DT, int N, int T, class X>
__device__ __forceinline__ void dot_rows(const uint16_t *const (&w)[N], const X &x, int rows, int K, float (&red)[4][N][T]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float acc[N][T];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[i][t] = 0.0f;
#pragma unroll 2
    for (int k = 512 * wave + 8 * lane; k < K; k += 2048) {
        u32x4 raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(w[i] + k));
        f32x8 xs[T];
#pragma unroll
        for (int t = 0; t < T; ++t) xs[t] = x(t < rows ? t : 0, k);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const f32x8 v = unpack8<DT>(raw[i]);
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[i][t] = __builtin_fmaf(v.v[e], xs[t].v[e], acc[i][t]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int o = 32; o; o >>= 1) acc[i][t] += __shfl_xor(acc[i][t], o);
            if (lane == 0) red[wave][i][t] = acc[i][t];
        }
    __syncthreads();
}
template <int N, int T>
__device__ __forceinline__ float joined(const float (&red)[4][N][T], int i, int t) {
    return ((red[0][i][t] + red[1][i][t]) + red[2][i][t]) + red[3][i][t];
}

}  // namespace tile
}  // namespace dgw
