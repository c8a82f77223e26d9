// loss_api.hip -- the C ABI declared in include/gemm_loss.h: argument checks,
// planning, workspace layout and kernel launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/gemm_loss.h"
#include "call.h"
#include "internal.h"
#include "loss.h"

namespace {

using namespace dgw::call;
using dgw::set_error;
using dgw::set_hip_error;

constexpr int64_t PIECE_BYTES = int64_t(256) << 20;   // the logits' gradient of one piece

int64_t row_of_w(const gemm_loss_args_t &a) { return (a.layout & 0xFu) == GEMM_B_NK ? a.H : a.V; }
int64_t rows_of_w(const gemm_loss_args_t &a) { return (a.layout & 0xFu) == GEMM_B_NK ? a.V : a.H; }

// What the host can tell from sizes, words and flags alone.
int check_sizes(const gemm_loss_args_t &a) {
    if (a.layout & ~0x1Fu || (a.layout & 0xEu)) return bad("layout word has unknown bits");
    if (a.kind > GEMM_LOSS_DISTILL) return bad("unknown kind of loss");
    if (a.T < 0 || a.V < 1 || a.H < 1) return bad("T >= 0, V >= 1 and H >= 1");
    if (a.T > GEMM_LOSS_MAX_T || a.V > GEMM_LOSS_MAX_V || a.H > GEMM_LOSS_MAX_H)
        return set_error(GEMM_ERR_UNSUPPORTED, "T, V or H exceeds GEMM_LOSS_MAX_T, GEMM_LOSS_MAX_V or GEMM_LOSS_MAX_H");
    if (a.T * a.V > GEMM_LOSS_MAX_TV || a.T * a.H > GEMM_LOSS_MAX_TH)
        return set_error(GEMM_ERR_UNSUPPORTED, "T * V or T * H exceeds GEMM_LOSS_MAX_TV or GEMM_LOSS_MAX_TH");
    if (a.H % 8) return set_error(GEMM_ERR_UNSUPPORTED, "H must be a multiple of 8");
    if ((a.layout & 0xFu) == GEMM_B_KN && a.V % 8)
        return set_error(GEMM_ERR_UNSUPPORTED, "V must be a multiple of 8 for GEMM_B_KN");
    if (a.kind == GEMM_LOSS_DISTILL) {
        if (a.entries < 1 || a.entries > GEMM_LOSS_MAX_ENTRIES) return bad("entries must be 1 .. GEMM_LOSS_MAX_ENTRIES");
        if (a.teacher_type > GEMM_LOSS_FP16) return bad("unknown type of the teacher's logits");
    }
    if (a.dw_type > GEMM_LOSS_DW_FP32_ADD) return bad("unknown dw_type");
    return GEMM_OK;
}

Blocks blocks_of(const gemm_loss_args_t &a, bool backward) {
    Blocks s;
    const int64_t t4 = a.T * 4, w_row = row_of_w(a) * 2, w_rows = rows_of_w(a);
    const int64_t dw_size = a.dw_type != GEMM_LOSS_DW_SAME ? 4 : 2;
    if (backward) {
        s.add(a.dx, a.T, a.H * 2, or_packed(a.lddx, a.H) * 2, "dx");
        s.add(a.dw, w_rows, row_of_w(a) * dw_size, or_packed(a.lddw, row_of_w(a)) * dw_size, "dw");
    } else {
        s.add(a.loss, 1, t4, t4, "loss");
        s.add(a.lse, 1, t4, t4, "lse");
    }
    s.written = s.all;
    s.add(a.x, a.T, a.H * 2, or_packed(a.ldx, a.H) * 2, "x");
    s.add(a.w, w_rows, w_row, or_packed(a.ldw, row_of_w(a)) * 2, "w");
    if (backward) {
        s.add(a.lse, 1, t4, t4, "lse");
        s.add(a.grad, 1, t4, t4, "grad");
    }
    if (a.kind == GEMM_LOSS_XENT) {
        s.add(a.target, 1, a.T * 8, a.T * 8, "target");
    } else {
        const int64_t n = a.T * a.entries, size = a.teacher_type == GEMM_LOSS_FP32 ? 4 : 2;
        s.add(a.teacher_index, 1, n * 8, n * 8, "teacher_index");
        s.add(a.teacher_logits, 1, n * size, n * size, "teacher_logits");
    }
    return s;
}

int check_args(const gemm_loss_args_t &a, bool backward) {
    int rc = check_sizes(a);
    if (rc != GEMM_OK) return rc;
    const int64_t ldx = or_packed(a.ldx, a.H), ldw = or_packed(a.ldw, row_of_w(a));
    if ((rc = check_ld(ldx, a.H, 8, "x")) != GEMM_OK || (rc = check_ld(ldw, row_of_w(a), 8, "w")) != GEMM_OK) return rc;
    if (a.kind == GEMM_LOSS_XENT && !(a.z_loss >= 0.0f && std::isfinite(a.z_loss))) return bad("z_loss must be finite and >= 0");
    if (a.kind == GEMM_LOSS_DISTILL) {
        const float square = a.temperature * a.temperature;
        if (!(a.temperature > 0.0f && square > 0.0f && std::isfinite(square)))
            return bad("temperature and its square must be finite and > 0");
    }
    if (a.num_cus < 0 || a.num_cus > MAX_CUS) return bad("num_cus must be 0 .. 65536");
    const bool dw32 = a.dw_type != GEMM_LOSS_DW_SAME;
    const int64_t lddx = or_packed(a.lddx, a.H), lddw = or_packed(a.lddw, row_of_w(a));
    if (backward) {
        if (a.dx && (rc = check_ld(lddx, a.H, 8, "dx")) != GEMM_OK) return rc;
        if (a.dw && (rc = check_ld(lddw, row_of_w(a), dw32 ? 4 : 8, "dw")) != GEMM_OK) return rc;
        if (a.dw && (reinterpret_cast<uintptr_t>(a.dw) & 15)) return set_error(GEMM_ERR_UNSUPPORTED, "dw must be 16-byte aligned");
    }
    if (a.T == 0) return apart(blocks_of(a, backward));   // a gradient of no rows is cleared
    if (!a.x || !a.w || !a.lse) return bad("x, w and lse must be non-null");
    if ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.dx)) & 15)
        return set_error(GEMM_ERR_UNSUPPORTED, "x, w and dx must be 16-byte aligned");
    if (a.kind == GEMM_LOSS_XENT ? !a.target : !a.teacher_index || !a.teacher_logits)
        return bad("the loss's targets must be non-null");
    if (a.workspace && reinterpret_cast<uintptr_t>(a.workspace) & 255) return bad("a caller workspace must be 256-byte aligned");
    if (!backward && !a.loss) return bad("loss must be non-null");
    if (backward && !a.grad) return bad("grad must be non-null");
    return apart(blocks_of(a, backward));
}

// Byte offsets of a call's parts in its workspace.
struct Layout {
    int64_t entries = 0, starts = 0, entropy = 0;  // the teacher's entries
    int64_t stats = 0;                            // forward
    int64_t scale = 0, dz = 0, dx = 0, dw = 0;    // backward
    int64_t ldd = 0, part = 0;                     // dz's rows, and from its first part to its second, in elements
    int64_t bytes = 0;
    int64_t take(int64_t n) {
        const int64_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
};

// The logits' tile.  Up to 64 rows the stream of w is the cost and thin tiles
// keep more of it in flight (V = 32768, H = 2048, T = 32: 35 us on 64 x 64 tiles,
// 43 us on 128 x 128); a vocabulary of fewer 64-entry tiles than CUs is cut finer
// (V = 8192, H = 1536, T = 1: 11.6 us on 32 x 32, 13.8 us on 64 x 64).  So are more
// rows where 128 x 128 tiles would leave half the CUs idle (V = 16000, H = 4096,
// T = 100: 54 us on 128 x 128, 44 us on 64 x 128).
int logits_tile(const gemm_loss_args_t &a, int64_t V, int cus) {
    const bool kn = (a.layout & 0xFu) == GEMM_B_KN;
    if (a.T > 64) {
        if (!kn && 2 * ceil_div(V, 128) * ceil_div(a.T, 128) <= cus) return dgw::LT_64x128;
        return choose(V, a.T, a.H, false, cus).tile;
    }
    if (kn) return a.T <= 32 ? dgw::LT_128x32 : dgw::LT_128x64;
    return a.T <= 32 && V < 64 * (int64_t)cus ? dgw::LT_32x32 : dgw::LT_64x64;
}

// dx's tile and slices.  Few rows: one workgroup a CU, which is what fits with dz in
// two parts (with one part two fitted and were slower, their slices add up more: V =
// 32768, H = 2048, T = 2: 16 slices 61 us for dz and dx together, 32 slices 68 us).
Choice dx_choice(const gemm_loss_args_t &a, int64_t V, int cus) {
    if (a.T > 64) return choose(a.H, a.T, V, true, cus);
    const int tile = a.T <= 32 ? dgw::LT_128x32 : dgw::LT_128x64;
    return {tile, (int)std::max<int64_t>(1, std::min<int64_t>(cus / ceil_div(a.H, 128), ceil_div(V, 64) / 8))};
}

struct Plan {
    int logits = dgw::LT_128x128, dx = dgw::LT_128x128, dw = dgw::LT_128x128;   // tiles
    int64_t piece = 0;
    int pieces = 0, dx_splits = 1, dw_splits = 1;
    bool dw_outer = false;   // dw by the kernel of few rows
    Layout at;
};

Plan make_plan(const gemm_loss_args_t &a, bool backward, int cus) {
    Plan p;
    Layout &l = p.at;
    if (a.kind == GEMM_LOSS_DISTILL) {
        l.entries = l.take(a.T * a.entries * (int64_t)sizeof(uint2));
        l.starts = l.take(a.T * dgw::LOSS_STARTS * 2);
        l.entropy = l.take(a.T * 4);
    }
    if (!backward) {
        p.logits = logits_tile(a, a.V, cus);
        l.stats = l.take(3 * ceil_div(a.V, dgw::loss_tile_shape(p.logits).p) * a.T * 4);
        return p;
    }
    const int64_t rows = std::max<int64_t>(a.T, 1), parts = a.T <= dgw::LOSS_FEW ? 2 : 1;   // of dz
    p.piece = std::min(round_up(a.V, 64), std::max<int64_t>(1024, PIECE_BYTES / (2 * parts) / rows / 1024 * 1024));
    // dw alone: dz is most of the workspace, and pieces cost it only launches.  Its
    // second part stays within the 4 (T + 256)(H + 256) bytes that a slice of dx takes at
    // most (64 x 50001 x 2048: pieces of 22528 entries, 110 us; T = 20: one piece, 80 us).
    if (parts == 2 && !a.dx) p.piece = std::min(p.piece, std::max<int64_t>(1024, 2 * (rows + 256) * (a.H + 256) / rows / 1024 * 1024));
    p.pieces = (int)ceil_div(a.V, p.piece);
    l.ldd = p.piece;
    l.scale = l.take(8);
    l.dz = l.take(a.T * l.ldd * 2 * parts);
    l.part = parts == 2 ? a.T * l.ldd : 0;
    const int64_t first = std::min(a.V, p.piece);
    p.logits = logits_tile(a, first, cus);
    if (a.dx) {
        const Choice c = dx_choice(a, first, cus);
        p.dx = c.tile;
        p.dx_splits = c.splits;
        if (p.dx_splits > 1 || p.pieces > 1) l.dx = l.take(dgw::loss_slots_bytes(p.dx, a.H, a.T, p.dx_splits));
    }
    if (a.dw) {
        const bool nk = (a.layout & 0xFu) == GEMM_B_NK;
        const int64_t rp = nk ? a.H : first, rq = nk ? first : a.H;
        p.dw_outer = parts == 2;
        if (!p.dw_outer) {
            const Choice c = choose(rp, rq, a.T, true, cus);
            p.dw = c.tile;
            p.dw_splits = c.splits;
        }
        if (p.dw_splits > 1) l.dw = l.take(dgw::loss_slots_bytes(p.dw, rp, rq, p.dw_splits));
    }
    return p;
}

// The workspace, the stream and the teacher's entries of a call.
struct Call {
    hipStream_t stream;
    void *ws = nullptr;
    std::unique_lock<std::mutex> lock;   // held for the whole call where ws is the library's
    int cus;
    int dtype;
    bool nk;
    Plan plan;
    dgw::LossTargets targets;
    const float *entropy = nullptr;
};

int begin(const gemm_loss_args_t &a, bool backward, Call *c) {
    c->stream = dgw::call_stream(a.stream);
    c->dtype = (a.layout & 0xF0u) == GEMM_FP16 ? 1 : 0;
    c->nk = (a.layout & 0xFu) == GEMM_B_NK;
    int rc;
    c->cus = a.num_cus;
    if (!c->cus && (rc = dgw::current_device_cus(&c->cus)) != GEMM_OK) return rc;
    c->plan = make_plan(a, backward, c->cus);
    const Layout &l = c->plan.at;
    c->ws = a.workspace;
    if (a.workspace) {
        if ((int64_t)a.workspace_bytes < l.bytes)
            return set_error(GEMM_ERR_WORKSPACE, "caller workspace is smaller than plan.workspace_bytes (" + std::to_string(l.bytes) + ")");
        const Blocks s = blocks_of(a, backward);
        const Block ws{a.workspace, 1, l.bytes, l.bytes, "workspace"};
        for (int i = 0; i < s.all; ++i)
            if (overlap(ws, s.b[i])) return overlapping(ws, s.b[i]);
    } else if ((rc = dgw::library_workspace(l.bytes, c->stream, &c->ws, &c->lock)) != GEMM_OK) {
        return rc;
    }
    if (a.kind == GEMM_LOSS_XENT) {
        c->targets = {a.target, nullptr, nullptr, 0, 0};
        return GEMM_OK;
    }
    uint2 *entries = part<uint2>(c->ws, l.entries);
    uint16_t *starts = part<uint16_t>(c->ws, l.starts);
    float *entropy = part<float>(c->ws, l.entropy);
    const hipError_t e = dgw::launch_loss_teacher(a.T, a.entries, a.V, a.teacher_index, a.teacher_logits, a.teacher_type,
                                                  a.temperature, entries, starts, entropy, c->stream);
    if (e != hipSuccess) return set_hip_error(e, "launch the teacher's softmax");
    c->targets = {nullptr, entries, starts, a.entries, dgw::loss_bucket_width(a.V)};
    c->entropy = entropy;
    return GEMM_OK;
}

// The logits' problem over entries [v0, v0 + n).
dgw::LossProblem problem(const gemm_loss_args_t &a, const Call &c, int64_t v0, int64_t n) {
    dgw::LossProblem p;
    const int64_t ldw = or_packed(a.ldw, row_of_w(a));
    p.T = (int)a.T;
    p.V = (int)n;
    p.H = (int)a.H;
    p.c = 1.44269504088896340736f / (a.kind == GEMM_LOSS_DISTILL ? a.temperature : 1.0f);
    p.x = {static_cast<const uint16_t *>(a.x), or_packed(a.ldx, a.H), (int)a.T, true};
    p.w = {static_cast<const uint16_t *>(a.w) + (c.nk ? v0 * ldw : v0), ldw, (int)n, c.nk};
    p.v0 = v0;
    p.targets = c.targets;
    return p;
}

int forward(const gemm_loss_args_t &a) {
    dgw::clear_error();
    int rc = check_args(a, false);
    if (rc != GEMM_OK || a.T == 0) return rc;
    Call c;
    if ((rc = begin(a, false, &c)) != GEMM_OK) return rc;
    const int tiles = (int)ceil_div(a.V, dgw::loss_tile_shape(c.plan.logits).p);
    float *st = part<float>(c.ws, c.plan.at.stats);
    const dgw::LossStats s{st, st + tiles * a.T, st + 2 * tiles * a.T};
    hipError_t e = dgw::launch_loss_stats(c.dtype, c.plan.logits, problem(a, c, 0, a.V), s, c.stream);
    if (e != hipSuccess) return set_hip_error(e, "launch the logits' statistics");
    if ((e = dgw::launch_loss_finish(a, tiles, s, c.entropy, c.stream)) != hipSuccess) return set_hip_error(e, "launch the losses");
    return GEMM_OK;
}

int backward(const gemm_loss_args_t &a) {
    dgw::clear_error();
    int rc = check_args(a, true);
    if (rc != GEMM_OK || (!a.dx && !a.dw)) return rc;
    const int64_t ldw = or_packed(a.ldw, row_of_w(a)), lddx = or_packed(a.lddx, a.H), lddw = or_packed(a.lddw, row_of_w(a));
    const int dw_size = a.dw_type == GEMM_LOSS_DW_SAME ? 2 : 4;
    hipError_t e;
    if (a.T == 0) {
        if (!a.dw || a.dw_type == GEMM_LOSS_DW_FP32_ADD) return GEMM_OK;
        if ((e = dgw::launch_loss_zero(a.dw, rows_of_w(a), row_of_w(a) * dw_size, lddw * dw_size, dgw::call_stream(a.stream))) != hipSuccess)
            return set_hip_error(e, "zero dw");
        return GEMM_OK;
    }
    Call c;
    if ((rc = begin(a, true, &c)) != GEMM_OK) return rc;
    const Plan &pl = c.plan;
    const bool xent = a.kind == GEMM_LOSS_XENT;
    const float tau = xent ? 1.0f : a.temperature;
    const dgw::LossRows rows{a.V, a.z_loss, tau, 1.0f / tau, xent ? a.target : nullptr, a.ignore_index,
                             c.entropy, a.grad, a.lse};
    float *scale = c.dtype == 1 ? part<float>(c.ws, pl.at.scale) : nullptr;
    uint16_t *dz = part<uint16_t>(c.ws, pl.at.dz);
    if (scale && (e = dgw::launch_loss_scale(rows, a.T, scale, c.stream)) != hipSuccess) return set_hip_error(e, "launch dz's scale");
    const float *unscale = scale ? scale + 1 : nullptr;
    dgw::LossProduct px;
    for (int i = 0; i < pl.pieces; ++i) {
        const int64_t v0 = i * pl.piece, n = std::min(pl.piece, a.V - v0);
        const dgw::LossProblem p = problem(a, c, v0, n);
        if ((e = dgw::launch_loss_dz(c.dtype, pl.logits, p, rows, scale, dz, pl.at.ldd, pl.at.part, c.stream)) != hipSuccess)
            return set_hip_error(e, "launch the logits' gradient");
        if (a.dx) {   // dx[t][h] += sum_v w[v][h] dz[t][v]
            px.P = {p.w.base, ldw, (int)a.H, !c.nk};
            px.Q = {dz, pl.at.ldd, (int)a.T, true, pl.at.part};
            px.K = (int)n;
            px.splits = pl.dx_splits;
            px.unscale = unscale;
            px.out = a.dx;
            px.ldo = lddx;
            px.out_kind = dgw::LO_16;
            if (pl.dx_splits > 1 || pl.pieces > 1) {
                px.out = part<float>(c.ws, pl.at.dx);
                px.out_kind = i == 0 ? dgw::LO_SLOTS : dgw::LO_SLOTS_ADD;
            }
            if ((e = dgw::launch_loss_product(c.dtype, pl.dx, px, c.stream)) != hipSuccess) return set_hip_error(e, "launch dx");
        }
        if (a.dw) {   // dw[v][h] = sum_t x[t][h] dz[t][v], as stored
            const dgw::LossMatrix mx{static_cast<const uint16_t *>(a.x), or_packed(a.ldx, a.H), (int)a.H, false};
            const dgw::LossMatrix mz{dz, pl.at.ldd, (int)n, false, pl.at.part};
            dgw::LossProduct q;
            q.P = c.nk ? mx : mz;
            q.Q = c.nk ? mz : mx;
            q.K = (int)a.T;
            q.splits = pl.dw_splits;
            q.unscale = unscale;
            q.out = static_cast<char *>(a.dw) + (c.nk ? v0 * lddw : v0) * dw_size;
            q.ldo = lddw;
            q.out_kind = a.dw_type == GEMM_LOSS_DW_SAME ? dgw::LO_16 : a.dw_type == GEMM_LOSS_DW_FP32 ? dgw::LO_F32 : dgw::LO_F32_ADD;
            const dgw::LossProduct join = q;
            if (pl.dw_splits > 1) {
                q.out = part<float>(c.ws, pl.at.dw);
                q.out_kind = dgw::LO_SLOTS;
            }
            if (pl.dw_outer) e = dgw::launch_loss_outer(c.dtype, q, 2 * c.cus, c.stream);
            else e = dgw::launch_loss_product(c.dtype, pl.dw, q, c.stream);
            if (e != hipSuccess) return set_hip_error(e, "launch dw");
            if (pl.dw_splits > 1 &&
                (e = dgw::launch_loss_join(c.dtype, pl.dw, join, part<float>(c.ws, pl.at.dw), c.stream)) != hipSuccess)
                return set_hip_error(e, "launch dw's join");
        }
    }
    if (a.dx && (pl.dx_splits > 1 || pl.pieces > 1)) {
        px.out = a.dx;
        px.out_kind = dgw::LO_16;
        if ((e = dgw::launch_loss_join(c.dtype, pl.dx, px, part<float>(c.ws, pl.at.dx), c.stream)) != hipSuccess)
            return set_hip_error(e, "launch dx's join");
    }
    return GEMM_OK;
}

int plan(const gemm_loss_args_t *args, int32_t backward, int32_t num_cus, gemm_loss_plan_t *out) {
    dgw::clear_error();
    if (!args || !out) return bad("args and out must be non-null");
    if (num_cus < 1 || num_cus > MAX_CUS) return bad("num_cus must be 1 .. 65536");
    const int rc = check_sizes(*args);
    if (rc != GEMM_OK) return rc;
    std::memset(out, 0, sizeof *out);
    const Plan p = make_plan(*args, backward != 0, num_cus);
    const dgw::LossTileShape l = dgw::loss_tile_shape(p.logits), x = dgw::loss_tile_shape(p.dx), w = dgw::loss_tile_shape(p.dw);
    out->tile_v = l.p;
    out->tile_t = l.q;
    out->num_cus = num_cus;
    out->workspace_bytes = p.at.bytes;
    if (backward) {
        out->pieces = p.pieces;
        out->piece = p.piece;
        out->dx_tile_h = x.p;
        out->dx_tile_t = x.q;
        out->dx_splits = p.dx_splits;
        out->dw_tile_p = w.p;
        out->dw_tile_q = w.q;
        out->dw_splits = p.dw_splits;
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_loss_plan(const gemm_loss_args_t *args, int32_t backward, int32_t num_cus, gemm_loss_plan_t *out) {
    return guarded([&] { return plan(args, backward, num_cus, out); });
}

int gemm_loss_forward(const gemm_loss_args_t *args) {
    return guarded([&] { return args ? forward(*args) : bad("args is null"); });
}

int gemm_loss_backward(const gemm_loss_args_t *args) {
    return guarded([&] { return args ? backward(*args) : bad("args is null"); });
}

}  // extern "C"
