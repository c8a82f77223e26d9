// ffn_api.hip -- the C ABI declared in include/gemm_ffn.h: argument checks,
// planning, workspace layout and kernel launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/gemm_ffn.h"
#include "call.h"
#include "ffn.h"
#include "internal.h"

namespace {

using namespace dgw::call;
using dgw::set_error;
using dgw::set_hip_error;

bool is_nk(const gemm_ffn_args_t &a) { return (a.layout & 0xFu) == GEMM_B_NK; }

// A weight as stored: rows and the row's length.
struct Shape {
    int64_t rows, row;
};
Shape shape_in(const gemm_ffn_args_t &a) { return is_nk(a) ? Shape{a.F, a.H} : Shape{a.H, a.F}; }     // w_gate, w_up
Shape shape_down(const gemm_ffn_args_t &a) { return is_nk(a) ? Shape{a.H, a.F} : Shape{a.F, a.H}; }

int check_sizes(const gemm_ffn_args_t &a) {
    if (a.layout & ~0x1Fu || (a.layout & 0xEu)) return bad("layout word has unknown bits");
    if (a.act > GEMM_FFN_RELU) return bad("unknown activation");
    if (a.T < 0 || a.H < 1 || a.F < 1) return bad("T >= 0, H >= 1 and F >= 1");
    if (a.T > GEMM_FFN_MAX_T || a.H > GEMM_FFN_MAX_H || a.F > GEMM_FFN_MAX_F)
        return set_error(GEMM_ERR_UNSUPPORTED, "T, H or F exceeds GEMM_FFN_MAX_T, GEMM_FFN_MAX_H or GEMM_FFN_MAX_F");
    if (a.T * a.H > GEMM_FFN_MAX_TH || a.T * a.F > GEMM_FFN_MAX_TH || a.H * a.F > GEMM_FFN_MAX_TH)
        return set_error(GEMM_ERR_UNSUPPORTED, "T * H, T * F or H * F exceeds GEMM_FFN_MAX_TH");
    if (a.H % 8 || a.F % 8) return set_error(GEMM_ERR_UNSUPPORTED, "H and F must be multiples of 8");
    if (a.dw_type > GEMM_FFN_DW_FP32_ADD) return bad("unknown dw_type");
    return GEMM_OK;
}

int dw_size(const gemm_ffn_args_t &a) { return a.dw_type == GEMM_FFN_DW_SAME ? 2 : 4; }

Blocks blocks_of(const gemm_ffn_args_t &a, bool backward) {
    Blocks s;
    const Shape in = shape_in(a), down = shape_down(a);
    // strides that check_ld refuses stay so in bytes, which could pass 64 bits
    auto stride = [](int64_t ld, int64_t row) { return std::clamp(or_packed(ld, row), int64_t(-1), MAX_LD + 1); };
    auto rows16 = [&](const void *p, int64_t rows, int64_t row, int64_t ld, const char *name) {
        s.add(p, rows, row * 2, stride(ld, row) * 2, name);
    };
    auto grad = [&](const void *p, Shape w, int64_t ld, const char *name) {
        s.add(p, w.rows, w.row * dw_size(a), stride(ld, w.row) * dw_size(a), name);
    };
    if (backward) {
        rows16(a.dx, a.T, a.H, a.lddx, "dx");
        grad(a.dw_gate, in, a.lddw_gate, "dw_gate");
        grad(a.dw_up, in, a.lddw_up, "dw_up");
        grad(a.dw_down, down, a.lddw_down, "dw_down");
    } else {
        rows16(a.y, a.T, a.H, a.ldy, "y");
        rows16(a.gate, a.T, a.F, a.ldgate, "gate");
        rows16(a.up, a.T, a.F, a.ldup, "up");
    }
    s.written = s.all;
    rows16(a.x, a.T, a.H, a.ldx, "x");
    rows16(a.w_gate, in.rows, in.row, a.ldw_gate, "w_gate");
    rows16(a.w_up, in.rows, in.row, a.ldw_up, "w_up");
    rows16(a.w_down, down.rows, down.row, a.ldw_down, "w_down");
    if (backward) {
        rows16(a.dy, a.T, a.H, a.lddy, "dy");
        rows16(a.gate, a.T, a.F, a.ldgate, "gate");
        rows16(a.up, a.T, a.F, a.ldup, "up");
    }
    return s;
}

int check_args(const gemm_ffn_args_t &a, bool backward) {
    int rc = check_sizes(a);
    if (rc != GEMM_OK) return rc;
    if (a.num_cus < 0 || a.num_cus > MAX_CUS) return bad("num_cus must be 0 .. 65536");
    const Blocks s = blocks_of(a, backward);
    const int unit32 = 4;
    for (int i = 0; i < s.all; ++i) {
        const Block &b = s.b[i];
        if (!b.base) continue;
        const bool fp32 = backward && i > 0 && i < s.written && dw_size(a) == 4;
        const int64_t size = fp32 ? 4 : 2;
        if ((rc = check_ld(b.ld / size, b.row / size, fp32 ? unit32 : 8, b.name)) != GEMM_OK) return rc;
        if (b.begin() & 15) return set_error(GEMM_ERR_UNSUPPORTED, std::string(b.name) + " must be 16-byte aligned");
    }
    if (a.T == 0) return apart(s);   // a gradient of no rows is cleared
    if (!a.x || !a.w_gate || !a.w_up || !a.w_down) return bad("x, w_gate, w_up and w_down must be non-null");
    if (!backward && !a.y) return bad("y must be non-null");
    if (!backward && !a.gate != !a.up) return bad("gate and up are kept both or neither");
    if (backward && (!a.dy || !a.gate || !a.up)) return bad("dy, gate and up must be non-null");
    if (a.workspace && reinterpret_cast<uintptr_t>(a.workspace) & 255) return bad("a caller workspace must be 256-byte aligned");
    return apart(s);
}

// Tile of the kernel that makes h from x.  Its P rows are both matrices' features.
int gate_tile(const gemm_ffn_args_t &a, int cus) {
    if (a.T > dgw::LOSS_FEW) return choose(2 * a.F, a.T, a.H, false, cus).tile;
    if (!is_nk(a)) return a.T <= 32 ? dgw::LT_128x32 : dgw::LT_128x64;
    return a.T <= 32 && a.F < 32 * (int64_t)cus ? dgw::LT_32x32 : dgw::LT_64x64;
}

int slope_tile(const gemm_ffn_args_t &a, int cus) {
    return a.T > dgw::LOSS_FEW ? choose(a.F, a.T, a.H, false, cus).tile : dgw::LT_64x64;
}

// Tile and slices of y and dx, products over k = F and 2 F features.  Few rows: one workgroup
// a CU, as two parts of h or dg leave room for.
Choice out_choice(const gemm_ffn_args_t &a, int64_t k, int cus) {
    if (a.T > dgw::LOSS_FEW) return choose(a.H, a.T, k, true, cus);
    const int tile = a.T <= 32 ? dgw::LT_128x32 : dgw::LT_128x64;
    return {tile, (int)std::max<int64_t>(1, std::min<int64_t>(cus / ceil_div(a.H, 128), ceil_div(k, 64) / 8))};
}

// Tile and slices of the rows of the weights' gradients, which one launch computes: by
// choose()'s model for their tiles together.
Choice weights_choice(const gemm_ffn_args_t &a, int cus) {
    const int64_t k = std::max<int64_t>(a.T, 1), each = (a.dw_gate ? 1 : 0) + (a.dw_up ? 1 : 0) + (a.dw_down ? 1 : 0);
    if (!each) return {dgw::LT_128x128, 1};
    // as one weight of `each` times the features: the tiles' number is all that counts
    return choose(a.H, each * round_up(a.F, 256), k, true, cus);
}

struct Plan {
    bool vec = false;                       // forward, by the kernels of single rows
    int first = dgw::LT_128x128;
    Choice out{dgw::LT_128x128, 1};
    bool outer = false;      // the weights' gradients by the kernel of few rows
    Choice weights{dgw::LT_128x128, 1};
    int parts = 1;
    int64_t part = 0;                       // elements from a first part to its second
    int64_t h = 0, dg = 0, du = 0, slots = 0;   // byte offsets
    int64_t bytes = 0;
    int64_t take(int64_t n) {
        const int64_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
};

Plan make_plan(const gemm_ffn_args_t &a, bool backward, int cus) {
    Plan p;
    p.parts = a.T <= dgw::LOSS_FEW ? 2 : 1;
    p.part = p.parts == 2 ? a.T * a.F : 0;
    const int64_t hidden = a.T * a.F * 2 * p.parts;
    int64_t slots = 0;
    auto need = [&](const Choice &c, int64_t rows_p, int64_t rows_q) {
        if (c.splits > 1) slots = std::max(slots, dgw::loss_slots_bytes(c.tile, rows_p, rows_q, c.splits));
    };
    p.h = p.take(hidden);   // two parts are as large as fp32
    p.vec = !backward && is_nk(a) && a.T <= dgw::FFN_VEC_T;
    if (p.vec) return p;
    p.out = out_choice(a, backward ? 2 * a.F : a.F, cus);
    if (!backward) {
        p.first = gate_tile(a, cus);
        need(p.out, a.H, a.T);
    } else {
        p.first = slope_tile(a, cus);
        p.dg = p.take(hidden);
        p.du = p.take(hidden);
        p.outer = a.T <= dgw::LOSS_FEW;
        if (!p.outer) {
            p.weights = weights_choice(a, cus);
            if (p.weights.splits > 1) {
                const Shape in = shape_in(a), down = shape_down(a);
                auto add = [&](const void *dw, Shape w) {
                    if (dw) slots += dgw::loss_slots_bytes(p.weights.tile, w.row, w.rows, p.weights.splits);
                };
                add(a.dw_gate, in);
                add(a.dw_up, in);
                add(a.dw_down, down);
            }
        }
        if (a.dx) {
            need(p.out, a.H, a.T);
            const int64_t packed = shape_in(a).row;
            if (or_packed(a.ldw_gate, packed) != or_packed(a.ldw_up, packed))
                slots = std::max(slots, dgw::loss_slots_bytes(p.out.tile, a.H, a.T, p.out.splits));
        }
    }
    if (slots) p.slots = p.take(slots);   // one product after the other
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
};

int begin(const gemm_ffn_args_t &a, bool backward, Call *c) {
    c->stream = dgw::call_stream(a.stream);
    c->dtype = (a.layout & 0xF0u) == GEMM_FP16 ? 1 : 0;
    c->nk = is_nk(a);
    int rc;
    c->cus = a.num_cus;
    if (!c->cus && (rc = dgw::current_device_cus(&c->cus)) != GEMM_OK) return rc;
    c->plan = make_plan(a, backward, c->cus);
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

dgw::LossMatrix matrix(const void *base, int64_t ld, int64_t packed, int64_t rows, bool kc, int64_t part = 0) {
    return {static_cast<const uint16_t *>(base), or_packed(ld, packed), (int)rows, kc, part};
}

// A product and, where its k is sliced, the slices' join.
int product(const Call &c, const Choice &how, dgw::LossProduct p, const char *what) {
    p.splits = how.splits;
    p.unscale = nullptr;
    const dgw::LossProduct join = p;
    float *slots = part<float>(c.ws, c.plan.slots);
    if (how.splits > 1) {
        p.out = slots;
        p.out_kind = dgw::LO_SLOTS;
    }
    hipError_t e = dgw::launch_loss_product(c.dtype, how.tile, p, c.stream);
    if (e == hipSuccess && how.splits > 1) e = dgw::launch_loss_join(c.dtype, how.tile, join, slots, c.stream);
    return e == hipSuccess ? GEMM_OK : set_hip_error(e, what);
}

int forward(const gemm_ffn_args_t &a) {
    dgw::clear_error();
    int rc = check_args(a, false);
    if (rc != GEMM_OK || a.T == 0) return rc;
    Call c;
    if ((rc = begin(a, false, &c)) != GEMM_OK) return rc;
    const Plan &pl = c.plan;
    const Shape in = shape_in(a), down = shape_down(a);
    uint16_t *h = part<uint16_t>(c.ws, pl.h);
    const dgw::FfnGate g{(int)a.T, (int)a.F, (int)a.H, matrix(a.w_gate, a.ldw_gate, in.row, a.F, c.nk),
                         matrix(a.w_up, a.ldw_up, in.row, a.F, c.nk), matrix(a.x, a.ldx, a.H, a.T, true), a.act,
                         h, a.F, pl.part, static_cast<uint16_t *>(a.gate), static_cast<uint16_t *>(a.up),
                         or_packed(a.ldgate, a.F), or_packed(a.ldup, a.F)};
    hipError_t e;
    if (pl.vec) {
        e = dgw::launch_ffn_vec(c.dtype, g, matrix(a.w_down, a.ldw_down, down.row, a.H, true), part<float>(c.ws, pl.h),
                                static_cast<uint16_t *>(a.y), or_packed(a.ldy, a.H), c.stream);
        return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch the block of single rows");
    }
    if ((e = dgw::launch_ffn_gate(c.dtype, pl.first, g, c.stream)) != hipSuccess) return set_hip_error(e, "launch the gated product");
    dgw::LossProduct y;   // y[t][o] = sum_f w_down[o][f] h[t][f]
    y.P = matrix(a.w_down, a.ldw_down, down.row, a.H, c.nk);
    y.Q = matrix(h, 0, a.F, a.T, true, pl.part);
    y.K = (int)a.F;
    y.out = a.y;
    y.ldo = or_packed(a.ldy, a.H);
    y.out_kind = dgw::LO_16;
    return product(c, pl.out, y, "launch y");
}

// The weights' gradients: `outs` holds a weight's output features, `ins` its input ones.
struct Weight {
    void *dw;
    int64_t ldo;
    dgw::LossMatrix outs, ins;
};
int weight_gradients(const gemm_ffn_args_t &a, const Call &c, const Weight (&w)[3]) {
    const int kind = a.dw_type == GEMM_FFN_DW_SAME ? dgw::LO_16 : a.dw_type == GEMM_FFN_DW_FP32 ? dgw::LO_F32 : dgw::LO_F32_ADD;
    hipError_t e;
    if (!c.plan.outer) {
        const Choice &how = c.plan.weights;
        dgw::FfnWeights p;
        p.T = (int)a.T;
        p.out_kind = kind;
        p.splits = how.splits;
        p.slots = how.splits > 1 ? part<float>(c.ws, c.plan.slots) : nullptr;
        for (int i = 0; i < 3; ++i) p.one[i] = {c.nk ? w[i].ins : w[i].outs, c.nk ? w[i].outs : w[i].ins, w[i].dw, w[i].ldo};
        e = dgw::launch_ffn_weights(c.dtype, how.tile, p, c.stream);
        return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch the weights' gradients");
    }
    dgw::LossProduct p[3];
    for (int i = 0; i < 3; ++i) {
        p[i].P = c.nk ? w[i].ins : w[i].outs;
        p[i].Q = c.nk ? w[i].outs : w[i].ins;
        p[i].K = (int)a.T;
        p[i].splits = 1;
        p[i].unscale = nullptr;
        p[i].out = w[i].dw;
        p[i].ldo = w[i].ldo;
        p[i].out_kind = kind;
    }
    e = dgw::launch_loss_outers(c.dtype, p, 2 * c.cus, c.stream);
    return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch the weights' gradients");
}

// dx[t][i] = sum_f w_gate[f][i] dg[t][f] + w_up[f][i] du[t][f].
int input_gradient(const gemm_ffn_args_t &a, const Call &c, const uint16_t *dg, const uint16_t *du) {
    const Plan &pl = c.plan;
    const Shape in = shape_in(a);
    const dgw::LossMatrix gate = matrix(a.w_gate, a.ldw_gate, in.row, a.H, !c.nk), up = matrix(a.w_up, a.ldw_up, in.row, a.H, !c.nk);
    const dgw::LossMatrix mg = matrix(dg, 0, a.F, a.T, true, pl.part), mu = matrix(du, 0, a.F, a.T, true, pl.part);
    dgw::LossProduct x;
    x.P = gate;
    x.Q = mg;
    x.K = (int)a.F;
    x.splits = pl.out.splits;
    x.out = a.dx;
    x.ldo = or_packed(a.lddx, a.H);
    x.out_kind = dgw::LO_16;
    x.unscale = nullptr;
    float *slots = part<float>(c.ws, pl.slots);
    hipError_t e;
    if (gate.ld == up.ld) {
        const dgw::FfnSum s{gate, up, mg, mu, (int)a.F, x.splits, x.splits > 1 ? static_cast<void *>(slots) : a.dx, x.ldo};
        e = dgw::launch_ffn_sum(c.dtype, pl.out.tile, s, c.stream);
    } else {   // weights of two strides: one product after the other, through the slots
        dgw::LossProduct one = x;
        one.out = slots;
        one.out_kind = dgw::LO_SLOTS;
        if ((e = dgw::launch_loss_product(c.dtype, pl.out.tile, one, c.stream)) != hipSuccess) return set_hip_error(e, "launch dx");
        one.P = up;
        one.Q = mu;
        one.out_kind = dgw::LO_SLOTS_ADD;
        e = dgw::launch_loss_product(c.dtype, pl.out.tile, one, c.stream);
    }
    if (e == hipSuccess && (x.splits > 1 || gate.ld != up.ld)) e = dgw::launch_loss_join(c.dtype, pl.out.tile, x, slots, c.stream);
    return e == hipSuccess ? GEMM_OK : set_hip_error(e, "launch dx");
}

int backward(const gemm_ffn_args_t &a) {
    dgw::clear_error();
    int rc = check_args(a, true);
    if (rc != GEMM_OK || (!a.dx && !a.dw_gate && !a.dw_up && !a.dw_down)) return rc;
    const Shape in = shape_in(a), down = shape_down(a);
    hipError_t e;
    if (a.T == 0) {
        if (a.dw_type == GEMM_FFN_DW_FP32_ADD) return GEMM_OK;
        auto zero = [&](void *dw, Shape w, int64_t ld) {
            return dw ? dgw::launch_loss_zero(dw, w.rows, w.row * dw_size(a), or_packed(ld, w.row) * dw_size(a), dgw::call_stream(a.stream))
                      : hipSuccess;
        };
        if ((e = zero(a.dw_gate, in, a.lddw_gate)) != hipSuccess || (e = zero(a.dw_up, in, a.lddw_up)) != hipSuccess ||
            (e = zero(a.dw_down, down, a.lddw_down)) != hipSuccess)
            return set_hip_error(e, "zero the weights' gradients");
        return GEMM_OK;
    }
    Call c;
    if ((rc = begin(a, true, &c)) != GEMM_OK) return rc;
    const Plan &pl = c.plan;
    uint16_t *h = part<uint16_t>(c.ws, pl.h), *dg = part<uint16_t>(c.ws, pl.dg), *du = part<uint16_t>(c.ws, pl.du);
    // w_down's features: stored [H,F] (nk) they are contiguous, [F,H] (kn) k is
    const dgw::FfnSlope s{(int)a.T, (int)a.F, (int)a.H, matrix(a.w_down, a.ldw_down, down.row, a.F, !c.nk),
                          matrix(a.dy, a.lddy, a.H, a.T, true), a.act,
                          static_cast<const uint16_t *>(a.gate), static_cast<const uint16_t *>(a.up),
                          or_packed(a.ldgate, a.F), or_packed(a.ldup, a.F), dg, du, h, a.F, pl.part};
    if ((e = dgw::launch_ffn_slope(c.dtype, pl.first, s, c.stream)) != hipSuccess) return set_hip_error(e, "launch the gates' gradients");
    if (a.dx && (rc = input_gradient(a, c, dg, du)) != GEMM_OK) return rc;
    const dgw::LossMatrix mx = matrix(a.x, a.ldx, a.H, a.H, false), mdy = matrix(a.dy, a.lddy, a.H, a.H, false);
    const dgw::LossMatrix mg = matrix(dg, 0, a.F, a.F, false, pl.part), mu = matrix(du, 0, a.F, a.F, false, pl.part),
                          mh = matrix(h, 0, a.F, a.F, false, pl.part);
    const Weight w[3] = {{a.dw_gate, or_packed(a.lddw_gate, in.row), mg, mx},
                         {a.dw_up, or_packed(a.lddw_up, in.row), mu, mx},
                         {a.dw_down, or_packed(a.lddw_down, down.row), mdy, mh}};
    return weight_gradients(a, c, w);
}

int plan(const gemm_ffn_args_t *args, int32_t backward, int32_t num_cus, gemm_ffn_plan_t *out) {
    dgw::clear_error();
    if (!args || !out) return bad("args and out must be non-null");
    if (num_cus < 1 || num_cus > MAX_CUS) return bad("num_cus must be 1 .. 65536");
    const int rc = check_sizes(*args);
    if (rc != GEMM_OK) return rc;
    std::memset(out, 0, sizeof *out);
    const Plan p = make_plan(*args, backward != 0, num_cus);
    const dgw::LossTileShape f = dgw::loss_tile_shape(p.first), o = dgw::loss_tile_shape(p.out.tile);
    out->num_cus = num_cus;
    out->workspace_bytes = p.bytes;
    if (p.vec) {   // four features or outputs a workgroup, every row; h in fp32
        out->first_tile_f = out->out_tile_h = 4;
        out->first_tile_t = out->out_tile_t = (int32_t)args->T;
        out->out_splits = 1;
        return GEMM_OK;
    }
    out->parts = p.parts;
    out->first_tile_f = backward ? f.p : f.p / 2;
    out->first_tile_t = f.q;
    out->out_tile_h = o.p;
    out->out_tile_t = o.q;
    out->out_splits = p.out.splits;
    if (backward) {
        const dgw::LossTileShape w = dgw::loss_tile_shape(p.weights.tile);
        out->dw_tile_p = w.p;
        out->dw_tile_q = w.q;
        out->dw_splits = p.weights.splits;
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_ffn_plan(const gemm_ffn_args_t *args, int32_t backward, int32_t num_cus, gemm_ffn_plan_t *out) {
    return guarded([&] { return plan(args, backward, num_cus, out); });
}

int gemm_ffn_forward(const gemm_ffn_args_t *args) {
    return guarded([&] { return args ? forward(*args) : bad("args is null"); });
}

int gemm_ffn_backward(const gemm_ffn_args_t *args) {
    return guarded([&] { return args ? backward(*args) : bad("args is null"); });
}

}  // extern "C"
