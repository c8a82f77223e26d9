// call.h -- what the C calls of the losses, the feed-forward block and the adapters
// share: checks of sizes, strides and overlaps, the choice of a product's tile
// (internal to the library).
#pragma once

#include <algorithm>
#include <cstdint>
#include <string>

#include "internal.h"
#include "loss.h"

namespace dgw {
namespace call {

constexpr int64_t MAX_LD = int64_t(1) << 21;   // a tile's rows then stay within 32-bit byte offsets
constexpr int MAX_CUS = 1 << 16;               // keeps a launch's workgroups within 32 bits

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

inline int64_t or_packed(int64_t ld, int64_t packed) { return ld ? ld : packed; }

inline int bad(const char *msg) { return set_error(GEMM_ERR_INVALID, msg); }

inline int check_ld(int64_t ld, int64_t row, int64_t unit, const char *what) {
    if (ld < row) return set_error(GEMM_ERR_INVALID, std::string(what) + ": rows overlap");
    if (ld % unit || ld > MAX_LD)
        return set_error(GEMM_ERR_UNSUPPORTED, std::string(what) + ": rows must start at multiples of 16 bytes, at most 2^21 elements apart");
    return GEMM_OK;
}

// A buffer of a call: `rows` rows of `row` bytes, `ld` bytes apart.
struct Block {
    const void *base;
    int64_t rows, row, ld;
    const char *name;
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(base); }
    uintptr_t end() const { return begin() + (uintptr_t)((rows - 1) * ld + row); }
};

inline bool overlap(const Block &a, const Block &b) {
    if (!a.base || !b.base || a.rows <= 0 || b.rows <= 0 || a.begin() >= b.end() || b.begin() >= a.end()) return false;
    if (a.ld != b.ld || a.rows == 1 || b.rows == 1) return true;
    // rows at one stride: each of a's begins `d` bytes behind where one of b's begins or would
    const uintptr_t ld = (uintptr_t)a.ld, d = (a.begin() % ld + ld - b.begin() % ld) % ld;
    return d < (uintptr_t)b.row || d + (uintptr_t)a.row > ld;
}

// The buffers of a call: first what it writes, then what it reads.
struct Blocks {
    Block b[16];
    int written = 0, all = 0;
    void add(const void *base, int64_t rows, int64_t row, int64_t ld, const char *name) { b[all++] = {base, rows, row, ld, name}; }
};

inline int overlapping(const Block &a, const Block &b) {
    return set_error(GEMM_ERR_INVALID, std::string(a.name) + " must not overlap " + b.name);
}

// What a call writes is apart from all else that it takes.
inline int apart(const Blocks &s) {
    for (int i = 0; i < s.written; ++i)
        for (int j = i + 1; j < s.all; ++j)
            if (overlap(s.b[i], s.b[j])) return overlapping(s.b[i], s.b[j]);
    return GEMM_OK;
}

// The tile of a product of rows_p x rows_q over k and, where its k may be sliced,
// the slices (of at least 8 slabs): the cheapest by a model of the time in us,
//   rounds of resident workgroups x (slabs x slab time + fixed time) + joining,
// for 256 x 256 tiles, one a CU (1.53 us a slab, 8 us fixed), and 128 x 128 tiles,
// two a CU (0.92 us a slab for the pair, 2.5 us fixed).  Model against measurement:
// logits of 333 x 50001 x 2048: 114 / 96 us (measured 97-106 / 92-96), of
// 200 x 50001 x 2048: 57 / 64 (58 / 67), of 777 x 50001 x 1536: 179 / 147 (150-166 /
// 143), of 500 x 32768 x 4096: 106 / 123 (111 / 143); dw of 500 x 32768 x 4096: 162 /
// 158 (154 / 158), of 2048 x 32768 x 2048: 228 / 255 (213 / 278); dx of
// 500 x 32768 x 4096: 124 / 130 (124 / 147), of 200 x 50001 x 2048: 61 / 56 (73 / 64).
// Joining takes a launch and reads the fp32 slices at 4.5 TB/s.
struct Choice {
    int tile, splits;
};
inline Choice choose(int64_t rows_p, int64_t rows_q, int64_t k, bool sliceable, int cus) {
    Choice best{dgw::LT_128x128, 1};
    double least = 0.0;
    const int64_t slabs = ceil_div(k, 64);
    auto consider = [&](int tile, double slab, double fixed) {
        const dgw::LossTileShape s = dgw::loss_tile_shape(tile);
        const int64_t tiles = ceil_div(rows_p, s.p) * ceil_div(rows_q, s.q), slots = (int64_t)cus * s.per_cu;
        const int64_t most = sliceable ? std::max<int64_t>(1, std::min<int64_t>(slots / tiles, slabs / 8)) : 1;
        for (int64_t n = 1; n <= most; ++n) {
            double us = (double)ceil_div(tiles * n, slots) * ((double)ceil_div(slabs, n) * slab + fixed);
            if (n > 1) us += 3.0 + 4.0 * (double)n * (double)rows_p * (double)rows_q / 4.5e6;
            if (least == 0.0 || us < least) {
                least = us;
                best = {tile, (int)n};
            }
        }
    };
    consider(dgw::LT_128x128, 0.92, 2.5);
    consider(dgw::LT_256x256, 1.53, 8.0);
    return best;
}

template <class T>
T *part(void *ws, int64_t at) {
    return reinterpret_cast<T *>(static_cast<char *>(ws) + at);
}

// No exception leaves a C call.  What can throw is the host's memory running out
// (an error's text is allocated); this text is short enough not to be.
template <class F>
int guarded(F &&f) noexcept {
    try {
        return f();
    } catch (...) {
        return set_error(GEMM_ERR_WORKSPACE, "no host memory");
    }
}

}  // namespace call
}  // namespace dgw
