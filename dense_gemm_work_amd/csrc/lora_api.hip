// lora_api.hip -- the C ABI declared in include/gemm_lora.h: argument checks,
// planning, workspace layout and kernel launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <string>
#include <utility>

#include "../../include/gemm_lora.h"
#include "call.h"
#include "internal.h"
#include "lora.h"

namespace {

using namespace dgw::call;
using dgw::set_error;
using dgw::set_hip_error;

bool is_nk(const gemm_lora_args_t &a) { return (a.layout & 0xFu) == GEMM_B_NK; }
int64_t w_rows(const gemm_lora_args_t &a) { return is_nk(a) ? a.N : a.H; }
int64_t w_row(const gemm_lora_args_t &a) { return is_nk(a) ? a.H : a.N; }
int64_t stride_a(const gemm_lora_args_t &a) { return or_packed(a.stride_a, (int64_t)a.R * a.H); }
int64_t stride_b(const gemm_lora_args_t &a) { return or_packed(a.stride_b, (int64_t)a.R * a.N); }
int dab_size(const gemm_lora_args_t &a) { return a.dab_type == GEMM_LORA_DAB_SAME ? 2 : 4; }

// Tiles of da and db: 64 of the rank by 128, for each adapter.
int64_t outer_tiles(const gemm_lora_args_t &a) {
    return a.adapters * ceil_div(a.R, 64) * ((a.da ? ceil_div(a.H, 128) : 0) + (a.db ? ceil_div(a.N, 128) : 0));
}

int check_sizes(const gemm_lora_args_t &a, bool backward) {
    if (a.layout & ~0x1Fu || (a.layout & 0xEu)) return bad("layout word has unknown bits");
    if (a.T < 0 || a.H < 1 || a.N < 1 || a.R < 1 || a.adapters < 1) return bad("T >= 0, H, N, R and adapters >= 1");
    if (a.T > GEMM_LORA_MAX_T || a.H > GEMM_LORA_MAX_H || a.N > GEMM_LORA_MAX_H || a.R > GEMM_LORA_MAX_R ||
        a.adapters > GEMM_LORA_MAX_ADAPTERS)
        return set_error(GEMM_ERR_UNSUPPORTED, "T, H, N, R or adapters exceeds its GEMM_LORA_MAX_*");
    if (a.T * a.H > GEMM_LORA_MAX_TH || a.T * a.N > GEMM_LORA_MAX_TH || a.H * a.N > GEMM_LORA_MAX_TH)
        return set_error(GEMM_ERR_UNSUPPORTED, "T * H, T * N or H * N exceeds GEMM_LORA_MAX_TH");
    if (a.adapters * (int64_t)a.R * std::max(a.H, a.N) > GEMM_LORA_MAX_LRH || (backward && a.adapters * a.T > GEMM_LORA_MAX_LT) ||
        a.T * a.R > GEMM_LORA_MAX_TR)
        return set_error(GEMM_ERR_UNSUPPORTED, "adapters * R * H, adapters * R * N, adapters * T or T * R exceeds its GEMM_LORA_MAX_*");
    if (backward && outer_tiles(a) > GEMM_LORA_MAX_TILES)
        return set_error(GEMM_ERR_UNSUPPORTED, "da and db have more than GEMM_LORA_MAX_TILES tiles; ask for them in two calls, or for fewer adapters");
    if (a.H % 8 || a.N % 8 || a.R % 8) return set_error(GEMM_ERR_UNSUPPORTED, "H, N and R must be multiples of 8");
    if (a.dab_type > GEMM_LORA_DAB_FP32_ADD) return bad("unknown dab_type");
    return GEMM_OK;
}

Blocks blocks_of(const gemm_lora_args_t &a, bool backward) {
    Blocks s;
    auto rows16 = [&](const void *p, int64_t rows, int64_t row, int64_t ld, const char *name) {
        s.add(p, rows, row * 2, or_packed(ld, row) * 2, name);
    };
    auto grad = [&](const void *p, int64_t n, const char *name) { s.add(p, 1, n * dab_size(a), n * dab_size(a), name); };
    const int64_t ra = (int64_t)a.R * a.H, rb = (int64_t)a.R * a.N;
    if (backward) {
        rows16(a.dx, a.T, a.H, a.lddx, "dx");
        grad(a.da, a.adapters * ra, "da");
        grad(a.db, a.adapters * rb, "db");
    } else {
        rows16(a.y, a.T, a.N, a.ldy, "y");
    }
    s.written = s.all;
    rows16(a.x, a.T, a.H, a.ldx, "x");
    rows16(a.w, w_rows(a), w_row(a), a.ldw, "w");
    rows16(a.a, a.adapters, ra, a.stride_a, "a");
    rows16(a.b, a.adapters, rb, a.stride_b, "b");
    if (backward) rows16(a.dy, a.T, a.N, a.lddy, "dy");
    s.add(a.adapter, 1, a.T * 8, a.T * 8, "adapter");
    s.add(a.scale, 1, a.adapters * 4, a.adapters * 4, "scale");
    return s;
}

int check_args(const gemm_lora_args_t &a, bool backward) {
    int rc = check_sizes(a, backward);
    if (rc != GEMM_OK) return rc;
    if (a.num_cus < 0 || a.num_cus > MAX_CUS) return bad("num_cus must be 0 .. 65536");
    if ((rc = check_ld(or_packed(a.ldx, a.H), a.H, 8, "x")) != GEMM_OK) return rc;
    if ((rc = check_ld(or_packed(a.ldw, w_row(a)), w_row(a), 8, "w")) != GEMM_OK) return rc;
    for (const auto &[stride, least] : {std::pair{stride_a(a), a.R * a.H}, std::pair{stride_b(a), a.R * a.N}})
        if (stride < least || stride % 8 || stride > GEMM_LORA_MAX_STRIDE)
            return bad("stride_a and stride_b must be at least a matrix, multiples of 8 and at most GEMM_LORA_MAX_STRIDE");
    if (!backward && (rc = check_ld(or_packed(a.ldy, a.N), a.N, 8, "y")) != GEMM_OK) return rc;
    if (backward && ((rc = check_ld(or_packed(a.lddy, a.N), a.N, 8, "dy")) != GEMM_OK ||
                     (rc = check_ld(or_packed(a.lddx, a.H), a.H, 8, "dx")) != GEMM_OK))
        return rc;
    const Blocks s = blocks_of(a, backward);
    for (int i = 0; i < s.all; ++i) {
        const uintptr_t unit = i == s.all - 1 ? 4 : i == s.all - 2 ? 8 : 16;   // scale, adapter, the matrices
        if (s.b[i].begin() & (unit - 1))
            return set_error(GEMM_ERR_UNSUPPORTED, std::string(s.b[i].name) + " must be " + std::to_string(unit) + "-byte aligned");
    }
    if (a.T == 0) return apart(s);   // a gradient of no rows is cleared
    if (!a.x || !a.w || !a.a || !a.b || !a.adapter) return bad("x, w, a, b and adapter must be non-null");
    if (!backward && !a.y) return bad("y must be non-null");
    if (backward && !a.dy) return bad("dy must be non-null");
    if (a.workspace && reinterpret_cast<uintptr_t>(a.workspace) & 255) return bad("a caller workspace must be 256-byte aligned");
    return apart(s);
}

// Few rows of small ranks with an adapter for at least every fourth of them: the narrow products
// row by row, as a tile of 64 rows would be read for one or two.  The gradients' call
// for 96 x 4096 x 4096, 64 adapters of rank 16: 46 us, on tiles 64; 200 x 2048 x 4096, 50
// of rank 32: 64 us, 77; its forward call 32 both ways; 250 x 4096 x 4096 with two of
// rank 16, which stays with the tiles: 25 us, row by row 27.5; 96 x 4096 x 4096 with 96 of
// rank 64, which does too: 97 and 122 us (gradients).  The pool's size stands for the
// adapters that the rows name, which the host does not know; a pool of 64 that rows name
// one of loses nothing by it: 200 x 4096 x 4096, rank 16, 26 us row by row and 30 on tiles
// (gradients 41 and 57; a pool of that one: 23 and 34).
bool low_by_rows(const gemm_lora_args_t &a) {
    return a.T <= dgw::LORA_FEW_T && a.R <= 32 && 4 * std::min<int64_t>(a.adapters, a.T) >= a.T;
}

// The narrow product's workgroups: over 64 rows, over the adapters among them and over
// slices of k.
struct Low {
    int lists = 1, splits = 1;
};
Low low_plan(const gemm_lora_args_t &a, int64_t k, bool kc, int cus) {
    const int64_t groups = ceil_div(std::max<int64_t>(a.T, 1), 64) * ceil_div(a.R, dgw::lora_low_rows(dgw::lora_low_tile(a.R, kc)));
    const int64_t most = std::min<int64_t>(a.adapters, std::min<int64_t>(std::max<int64_t>(a.T, 1), 64));
    // Few rows': one a CU, as the wide product's run beside them (96 x 4096 x 4096, 20 adapters
    // of rank 16: 19 us, with two 23; 96 of rank 64: 51 and 57).  More rows': two, of which
    // tiles of 64 ranks run one after the other, as one fits beside its list.
    const int64_t budget = a.T <= 256 ? cus : 2 * cus;
    Low l;
    l.lists = (int)std::max<int64_t>(1, std::min(most, budget / groups));
    // Beyond few rows a group has the one or two adapters of its requests, and the
    // workgroups that find none cost about what they wait for: at most four share a group's
    // adapters (the gradients' call for 1327 x 2536 x 5288 with 47 adapters of rank 8: 99 us, with 24
    // lists 136; 1000 x 2048 x 4096 with 64 mixed row by row: 254 us, eight lists 263, 24 lists
    // 328, two 273).  On both sides of few rows, x 4096 x 4096, rank 40, forward: 256 rows,
    // 64 mixed 61 us, with 24 lists 79, with four 258; 16 packed 32 from two lists on; 257 rows,
    // 64 mixed 83 in four and in 24 lists, 73 in six, 190 in one; 16 packed 36, in 24 lists 37.
    // Up to nine slices fill the CUs that few groups leave idle (x 4096 x 4096, four of rank 64:
    // 512 rows 41 us, in one slice 53, four 43, 16 46; gradients of 1024 rows 80, in one 87, four
    // 78, 16 91); many groups take two (gradients of 4096 rows 150, in one 154, four 161, nine
    // 182; of 8192 rows 283, 274, 303, 343; between them 2048 rows 106 in eight, 95 in two).
    if (a.T > 256) l.lists = std::min(l.lists, 4);
    const int64_t found = a.T <= 256 ? l.lists : std::min(l.lists, 2), most_splits = groups >= 64 ? 2 : 9;
    l.splits = (int)std::max<int64_t>(1, std::min({ceil_div(k, 64) / 2, budget / (groups * found), most_splits}));
    return l;
}

// The wide product's tile, and which of its tiles are computed whole and in how many
// slices the rest: the cheapest by choose()'s model of a tile's time (with 4 us more for the
// adapters) and of the join, for slices of every tile and for whole rounds of workgroups
// with slices of what is left over.  5000 x 4096 x 8192 on 256 CUs: 640 tiles of 256 x 256,
// the last 128 in two slices, 299 us in the model; in three rounds of whole tiles 330.
struct Wide {
    int tile = dgw::LP_128x128, splits = 1;
    int64_t whole = 0;   // tiles
};
int64_t tiles_of(int tile, int64_t rows_p, int64_t rows_q) {
    const dgw::LossTileShape s = dgw::lora_tile_shape(tile);
    return ceil_div(rows_p, s.p) * ceil_div(rows_q, s.q);
}
Wide out_plan(const gemm_lora_args_t &a, int64_t rows_p, int64_t k, bool few, int cus) {
    Wide best;
    const int64_t slabs = ceil_div(k, 64);
    if (a.T <= 128 || few) {
        best.tile = a.T <= 32 ? dgw::LP_64x32 : a.T <= 64 ? dgw::LP_64x64 : dgw::LP_64x128;
        // one workgroup a CU (96 x 4096 x 4096: 14.8 us, with two 16.2, and a shorter join)
        best.splits = (int)std::max<int64_t>(1, std::min(cus / (ceil_div(rows_p, 64) * std::max<int64_t>(1, ceil_div(a.T, 128))), slabs / 4));
        best.whole = best.splits == 1 ? tiles_of(best.tile, rows_p, a.T) : 0;
        return best;
    }
    double least = 0.0;
    auto consider = [&](int tile, double pair, double lone, double fixed) {
        const dgw::LossTileShape s = dgw::lora_tile_shape(tile);
        const int64_t tiles = tiles_of(tile, rows_p, a.T), slots = (int64_t)cus * s.per_cu;
        for (int64_t whole : {int64_t(0), tiles / slots * slots, tiles}) {
            const int64_t rest = tiles - whole;
            const int64_t most = rest ? std::max<int64_t>(1, std::min({slots / rest, slabs / 8, int64_t(16)})) : 1;
            for (int64_t n = 1; n <= most; ++n) {
                if (rest && whole && n == 1) continue;
                // a workgroup alone on its CU gets through its slabs faster
                const double slab = rest * n <= cus ? lone : pair;
                double us = (double)ceil_div(whole, slots) * ((double)slabs * pair + fixed);
                if (rest) us += (double)ceil_div(rest * n, slots) * ((double)ceil_div(slabs, n) * slab + fixed);
                if (rest && n > 1) us += 3.0 + 4.0 * (double)n * (double)rest * (double)(s.p * s.q) / 4.5e6;
                if (least == 0.0 || us < least) {
                    least = us;
                    best.tile = tile;
                    best.splits = (int)n;
                    best.whole = n == 1 ? tiles : whole;
                }
            }
        }
    };
    consider(dgw::LP_128x128, 0.92, 0.6, 6.5);
    consider(dgw::LP_256x256, 1.53, 1.53, 12.0);
    return best;
}

// Few rows of small ranks may take the adapters in the join, where each row reads its own
// adapter (R elements a result) whatever the other rows read; in the product's tiles each
// adapter costs about half a microsecond, and there are min(adapters, T) at most.  In the
// join, 238 x 296 x 6400 with 63 adapters of rank 24: 34 us, in the tiles 61; 96 x 4096 x
// 4096 with 64 of rank 16: 21 and 46; 256 x 8192 x 8192 with two of rank 32: 73 us, in the
// tiles 63.  Of a pool of 64 that the rows name one of (see low_by_rows): 200 x 4096 x 4096,
// rank 16, 26 us, in the tiles 40.
bool few_rows(const gemm_lora_args_t &a, int64_t wide) {
    if (a.T > dgw::LORA_FEW_T || a.R > dgw::LORA_FEW_R) return false;
    const double join = (double)(a.T * a.R) * (double)wide * 2.0 / 8e6;
    return join < 6.0 + 0.5 * (double)std::min<int64_t>(a.adapters, a.T);
}

// Slices of the rows for da and db, which one launch computes.
int outer_splits(const gemm_lora_args_t &a, int cus) {
    return (int)std::max<int64_t>(1, std::min(2 * cus / std::max<int64_t>(1, outer_tiles(a)), ceil_div(a.T, 64) / 8));
}

struct Plan {
    Low s, ds;
    Wide out;
    bool few = false, by_rows = false;
    int dab_splits = 1;
    int64_t db_at = 0;   // db's slices behind da's
    int64_t low = 0, dlow = 0, part_s = 0, part_ds = 0, slots = 0, partial = 0, masks = 0;   // byte offsets
    int64_t bytes = 0;
    int64_t take(int64_t n) {
        const int64_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
};

Plan make_plan(const gemm_lora_args_t &a, bool backward, int cus) {
    Plan p;
    const bool nk = is_nk(a);
    int64_t slots = 0;
    const bool own = backward && (a.da || a.db);   // the adapters' gradients: s and ds in the type, too
    auto low = [&](Low &l, int64_t k, bool kc, int64_t &slices, int64_t &at) {
        if (!p.by_rows) l = low_plan(a, k, kc, cus);
        slices = p.take(l.splits * a.T * a.R * 4);
        if (own) at = p.take(a.T * a.R * 2);
    };
    const int64_t wide = backward ? a.H : a.N;
    p.few = (!backward || a.dx) && few_rows(a, wide);
    p.by_rows = (backward || p.few) && low_by_rows(a);
    if (!backward || a.db) low(p.s, a.H, nk, p.part_s, p.low);
    if (backward && (a.dx || a.da)) low(p.ds, a.N, !nk, p.part_ds, p.dlow);
    if (!backward || a.dx) {
        p.out = out_plan(a, wide, backward ? a.N : a.H, p.few, cus);
        if (p.few) p.out.whole = 0;
        const dgw::LossTileShape s = dgw::lora_tile_shape(p.out.tile);
        slots = (tiles_of(p.out.tile, wide, a.T) - p.out.whole) * p.out.splits * s.p * s.q * 4;
    }
    if (slots) p.slots = p.take(slots);
    if (own) {
        p.masks = p.take(a.adapters * ceil_div(a.T, 64) * 8);
        p.dab_splits = outer_splits(a, cus);
        if (p.dab_splits > 1) {
            p.db_at = a.da ? round_up(p.dab_splits * (int64_t)a.adapters * a.R * a.H * 4, 256) : 0;
            p.partial = p.take(p.db_at + (a.db ? p.dab_splits * (int64_t)a.adapters * a.R * a.N * 4 : 0));
        }
    }
    return p;
}

struct Call {
    hipStream_t stream;
    void *ws = nullptr;
    std::unique_lock<std::mutex> lock;   // held for the whole call where ws is the library's
    int cus;
    int dtype;
    bool nk;
    Plan plan;
    dgw::LoraRows rows;
};

int begin(const gemm_lora_args_t &a, bool backward, Call *c) {
    c->stream = dgw::call_stream(a.stream);
    c->dtype = (a.layout & 0xF0u) == GEMM_FP16 ? 1 : 0;
    c->nk = is_nk(a);
    int rc;
    c->cus = a.num_cus;
    if (!c->cus && (rc = dgw::current_device_cus(&c->cus)) != GEMM_OK) return rc;
    c->plan = make_plan(a, backward, c->cus);
    c->rows = {a.adapter, (int)a.T, a.adapters, a.scale};
    c->ws = a.workspace;
    if (!a.workspace) return dgw::library_workspace(c->plan.bytes, c->stream, &c->ws, &c->lock);
    if ((int64_t)a.workspace_bytes < c->plan.bytes)
        return set_error(GEMM_ERR_WORKSPACE, "caller workspace is smaller than plan.workspace_bytes (" + std::to_string(c->plan.bytes) + ")");
    const Blocks s = blocks_of(a, backward);
    const Block ws{a.workspace, 1, c->plan.bytes, c->plan.bytes, "workspace"};
    for (int i = 0; i < s.all; ++i)
        if (overlap(ws, s.b[i])) return overlapping(ws, s.b[i]);
    return GEMM_OK;
}

dgw::LossMatrix matrix(const void *base, int64_t ld, int64_t packed, int64_t rows, bool kc) {
    dgw::LossMatrix m;
    m.base = static_cast<const uint16_t *>(base);
    m.ld = or_packed(ld, packed);
    m.rows = (int)rows;
    m.kc = kc;
    return m;
}

// a as `rows` x `k`: [R][H] (nk) or [H][R] (kn); b: [N][R] (nk) or [R][N] (kn).
dgw::LoraFactor factor_a(const gemm_lora_args_t &a, bool rank_rows) {   // rows: the rank, or H
    const bool nk = is_nk(a);
    return {matrix(a.a, 0, nk ? a.H : a.R, rank_rows ? a.R : a.H, rank_rows == nk), stride_a(a)};
}
dgw::LoraFactor factor_b(const gemm_lora_args_t &a, bool rank_rows) {   // rows: the rank, or N
    const bool nk = is_nk(a);
    return {matrix(a.b, 0, nk ? a.R : a.N, rank_rows ? a.R : a.N, rank_rows != nk), stride_b(a)};
}

dgw::LoraLow narrow(const gemm_lora_args_t &a, const Call &c, const Low &l, const dgw::LoraFactor &f, const dgw::LossMatrix &x, int64_t k,
                    int64_t slices) {
    return {c.rows, f, x, a.R, (int)k, l.lists, l.splits, part<float>(c.ws, slices), c.plan.by_rows};
}

dgw::LoraProduct product(const gemm_lora_args_t &a, const Call &c, const dgw::LossMatrix &w, const dgw::LossMatrix &x,
                         const dgw::LoraFactor &f, const dgw::LoraLow &low, int64_t k, void *out, int64_t ldo) {
    const Wide &o = c.plan.out;
    const bool sliced = o.splits > 1 || c.plan.few;
    return {c.rows, w, x, f, low.partial, low.splits, (int)k, a.R, o.splits, (int)o.whole,
            sliced ? part<float>(c.ws, c.plan.slots) : nullptr, out, ldo};
}

int forward(const gemm_lora_args_t &a) {
    dgw::clear_error();
    int rc = check_args(a, false);
    if (rc != GEMM_OK || a.T == 0) return rc;
    Call c;
    if ((rc = begin(a, false, &c)) != GEMM_OK) return rc;
    const dgw::LossMatrix x = matrix(a.x, a.ldx, a.H, a.T, true);
    const dgw::LoraLow s = narrow(a, c, c.plan.s, factor_a(a, true), x, a.H, c.plan.part_s);
    const dgw::LoraProduct y = product(a, c, matrix(a.w, a.ldw, w_row(a), a.N, c.nk), x, factor_b(a, false), s, a.H, a.y,
                                       or_packed(a.ldy, a.N));
    hipError_t e;
    if (c.plan.few) {
        e = dgw::launch_lora_few(c.dtype, c.plan.out.tile, y, s, c.stream);
        return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch the projection of few rows");
    }
    if ((e = dgw::launch_lora_low(c.dtype, s, c.stream)) != hipSuccess) return set_hip_error(e, "launch the narrow product");
    e = dgw::launch_lora_product(c.dtype, c.plan.out.tile, y, dgw::LoraLowJoin(), c.stream);
    if (e == hipSuccess && y.splits > 1) e = dgw::launch_lora_join(c.dtype, c.plan.out.tile, y, c.stream);
    return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch the projection");
}

// da or db: out[o][i] = sum over an adapter's rows of outs[t][o] ins[t][i] as "nk" stores
// it; one of them holds the narrow rows.
dgw::LoraOuter outer(const gemm_lora_args_t &a, const Call &c, const dgw::LossMatrix &outs, const dgw::LossMatrix &ins, bool narrow_ins,
                     int64_t at, void *out) {
    dgw::LoraOuter p;
    p.P = c.nk ? ins : outs;
    p.Q = c.nk ? outs : ins;
    p.narrow_p = narrow_ins == c.nk;
    p.T = (int)a.T;
    p.count = a.adapters;
    p.masks = part<uint64_t>(c.ws, c.plan.masks);
    p.splits = c.plan.dab_splits;
    p.partial = part<float>(c.ws, c.plan.partial + at);
    p.out_kind = a.dab_type == GEMM_LORA_DAB_SAME ? dgw::LO_16 : a.dab_type == GEMM_LORA_DAB_FP32 ? dgw::LO_F32 : dgw::LO_F32_ADD;
    p.out = out;
    p.ldo = p.P.rows;
    p.stride = (int64_t)p.P.rows * p.Q.rows;
    return p;
}

int backward(const gemm_lora_args_t &a) {
    dgw::clear_error();
    int rc = check_args(a, true);
    if (rc != GEMM_OK || (!a.dx && !a.da && !a.db)) return rc;
    hipError_t e;
    if (a.T == 0) {
        if (a.dab_type == GEMM_LORA_DAB_FP32_ADD) return GEMM_OK;
        auto zero = [&](void *p, int64_t row) {
            return p ? dgw::launch_loss_zero(p, (int64_t)a.adapters * a.R, row * dab_size(a), row * dab_size(a), dgw::call_stream(a.stream))
                     : hipSuccess;
        };
        if ((e = zero(a.da, a.H)) != hipSuccess || (e = zero(a.db, a.N)) != hipSuccess) return set_hip_error(e, "zero da and db");
        return GEMM_OK;
    }
    Call c;
    if ((rc = begin(a, true, &c)) != GEMM_OK) return rc;
    const Plan &pl = c.plan;
    const bool own = a.da || a.db;
    const dgw::LossMatrix x = matrix(a.x, a.ldx, a.H, a.T, true), dy = matrix(a.dy, a.lddy, a.N, a.T, true);
    dgw::LoraLow s = narrow(a, c, pl.s, factor_a(a, true), x, a.H, pl.part_s);
    dgw::LoraLow ds = narrow(a, c, pl.ds, factor_b(a, true), dy, a.N, pl.part_ds);
    if (!a.db) s.partial = nullptr;
    if (!a.dx && !a.da) ds.partial = nullptr;
    if ((e = dgw::launch_lora_lows(c.dtype, s, ds, own ? part<uint64_t>(c.ws, pl.masks) : nullptr, c.stream)) != hipSuccess)
        return set_hip_error(e, "launch the narrow products");
    dgw::LoraLowJoin join;
    if (own)
        join = {c.rows, a.R, s.partial, ds.partial, s.splits, ds.splits, s.partial ? part<uint16_t>(c.ws, pl.low) : nullptr,
                ds.partial ? part<uint16_t>(c.ws, pl.dlow) : nullptr};
    dgw::LoraProduct dx;
    if (a.dx) {
        dx = product(a, c, matrix(a.w, a.ldw, w_row(a), a.H, !c.nk), dy, factor_a(a, false), ds, a.N, a.dx, or_packed(a.lddx, a.H));
        if (pl.few) dx.partial = nullptr;
        e = dgw::launch_lora_product(c.dtype, pl.out.tile, dx, join, c.stream);
        if (e == hipSuccess && !own && pl.few) e = dgw::launch_lora_few_join(c.dtype, pl.out.tile, dx, ds, c.stream);
        else if (e == hipSuccess && !own && dx.splits > 1) e = dgw::launch_lora_join(c.dtype, pl.out.tile, dx, c.stream);
    } else {
        e = dgw::launch_lora_low_join(c.dtype, join, c.stream);
    }
    if (e != hipSuccess) return set_hip_error(e, "launch dx");
    if (!own) return GEMM_OK;
    const dgw::LossMatrix ms = matrix(join.s_low, 0, a.R, a.R, false), mds = matrix(join.ds_low, 0, a.R, a.R, false);
    const dgw::LossMatrix mx = matrix(a.x, a.ldx, a.H, a.H, false), mdy = matrix(a.dy, a.lddy, a.N, a.N, false);
    e = dgw::launch_lora_outers(c.dtype, outer(a, c, mds, mx, false, 0, a.da), outer(a, c, mdy, ms, true, pl.db_at, a.db),
                                pl.out.tile, a.dx && (dx.splits > 1 || pl.few) ? &dx : nullptr, pl.few ? &ds : nullptr, c.stream);
    return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch da and db");
}

int plan(const gemm_lora_args_t *args, int32_t backward, int32_t num_cus, gemm_lora_plan_t *out) {
    dgw::clear_error();
    if (!args || !out) return bad("args and out must be non-null");
    if (num_cus < 1 || num_cus > MAX_CUS) return bad("num_cus must be 1 .. 65536");
    const int rc = check_sizes(*args, backward != 0);
    if (rc != GEMM_OK) return rc;
    std::memset(out, 0, sizeof *out);
    const Plan p = make_plan(*args, backward != 0, num_cus);
    const bool kc = is_nk(*args) == !backward;
    const Low &l = backward ? p.ds : p.s;
    const dgw::LossTileShape o = dgw::lora_tile_shape(p.out.tile);
    out->num_cus = num_cus;
    out->low_tile_r = p.by_rows ? 8 : dgw::lora_low_rows(dgw::lora_low_tile(args->R, kc));
    out->low_splits = l.splits;
    out->low_lists = l.lists;
    out->out_tile_p = o.p;
    out->out_tile_t = o.q;
    out->out_splits = p.out.splits;
    out->out_whole = p.out.whole;
    if (backward) out->dab_splits = p.dab_splits;
    out->workspace_bytes = p.bytes;
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_lora_plan(const gemm_lora_args_t *args, int32_t backward, int32_t num_cus, gemm_lora_plan_t *out) {
    return guarded([&] { return plan(args, backward, num_cus, out); });
}

int gemm_lora_forward(const gemm_lora_args_t *args) {
    return guarded([&] { return args ? forward(*args) : bad("args is null"); });
}

int gemm_lora_backward(const gemm_lora_args_t *args) {
    return guarded([&] { return args ? backward(*args) : bad("args is null"); });
}

}  // extern "C"
