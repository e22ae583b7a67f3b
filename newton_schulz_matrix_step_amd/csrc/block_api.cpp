// Host side of the block operators (the gated feed-forward, the norms around a
// block, dropout): argument validation, workspaces and launches.  Each call
// validates everything before it enqueues anything.

#include "layer_host.hpp"

using namespace muon;

static_assert(int(MUON_GATE_SILU) == int(GATE_SILU) && int(MUON_GATE_GELU) == int(GATE_GELU) &&
                  int(MUON_GATE_SIGMOID) == int(GATE_SIGMOID) && int(MUON_GATE_RELU) == int(GATE_RELU),
              "gate codes");
static_assert(int(MUON_NORM_RMS) == int(NORM_RMS) && int(MUON_NORM_LAYER) == int(NORM_LAYER), "norm codes");

namespace {

muon_status run_gated(HandleBase* h, GatedArgs& a, hipStream_t stream) {
    if (gated_tiles128(a) > kMaxTiles128)
        return fail(h, MUON_ERR_INVALID_ARG, "more than %lld output tiles of 128 x 128", (long long)kMaxTiles128);
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    const GatedPlan p = plan_gated(a);
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    size_t at[7] = {0, p.partial_bytes, p.db_bytes, p.a_bytes, a.pair == PAIR_K ? p.a_bytes : 0, p.b_bytes,
                    a.pair != PAIR_NONE ? p.b_bytes : 0};
    for (int i = 1; i < 7; ++i) at[i] = at[i - 1] + up(at[i]);
    void* ws = nullptr;
    const muon_status st = workspace(h, at[6], stream, &ws);
    if (st != MUON_OK) return st;
    char* base = static_cast<char*>(ws);
    if (p.partial_bytes) a.partial = reinterpret_cast<float*>(base);
    if (p.db_bytes) a.db_partial = reinterpret_cast<float*>(base + at[1]);
    if (p.a_bytes) a.a_ws = base + at[2], a.a2_ws = base + at[3];
    if (p.b_bytes) a.b_ws = base + at[4], a.b2_ws = base + at[5];
    const hipError_t e = launch_gated(a, stream);
    if (e != hipSuccess) return hip_fail(h, e, "gated feed-forward launch");
    return MUON_OK;
}

bool pair_vec(const void* p, const void* q, int64_t ld, int32_t dtype) { return rows_vec(p, ld, dtype) && rows_vec(q, ld, dtype); }

// Both tensors of a pair of pre-activations, in full or in 8 bits.
void check_pair(Check& ck, const void* gate, const void* up, const muon_act8& gate8, const muon_act8& up8, int64_t ld_z,
                int64_t hidden, int32_t dtype) {
    ck.matrix(gate, ld_z, hidden, dtype, "gate");
    ck.matrix(up, ld_z, hidden, dtype, "up");
    ck.act8(gate8, hidden, "gate8");
    ck.act8(up8, hidden, "up8");
    ck.need((gate != nullptr) == (up != nullptr), "one of gate and up");
    ck.need((gate8.codes != nullptr) == (up8.codes != nullptr), "one of gate8 and up8");
    ck.need(!(gate && gate8.codes), "both gate and gate8");
}

muon_status gated_forward(muon_handle* handle, const muon_gated_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_gated_args& p = *args;
    ck.dtype(p.dtype, "x");
    if (p.bias_gate || p.bias_up) ck.dtype(p.bias_dtype, "bias");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.in, 1, kMaxCols, "in");
    ck.size(p.hidden, 1, kMaxCols, "hidden");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.activation >= MUON_GATE_SILU && p.activation <= MUON_GATE_RELU, "unknown activation %d", p.activation);
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || (p.x && p.h), "x or h is NULL");
    ck.need(p.w_gate && p.w_up, "w_gate or w_up is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN;
    ck.matrix(p.x, p.ld_x, p.in, p.dtype, "x");
    ck.matrix(p.w_gate, p.ld_w, oi ? p.in : p.hidden, p.dtype, "w_gate");
    ck.matrix(p.w_up, p.ld_w, oi ? p.in : p.hidden, p.dtype, "w_up");
    ck.matrix(p.h, p.ld_h, p.hidden, p.dtype, "h");
    ck.vector(p.bias_gate, p.bias_dtype, "bias_gate");
    ck.vector(p.bias_up, p.bias_dtype, "bias_up");
    check_pair(ck, p.gate, p.up, p.gate8, p.up8, p.ld_z, p.hidden, p.dtype);
    ck.distinct({p.h, p.gate, p.up, p.gate8.codes, p.gate8.exponents, p.up8.codes, p.up8.exponents},
                {p.x, p.w_gate, p.w_up, p.bias_gate, p.bias_up});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    GatedArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_GATED;
    a.pair = PAIR_COLS;
    a.gate_act = p.activation;
    a.a = p.x;
    a.b = p.w_gate;
    a.b2 = p.w_up;
    a.lda = p.ld_x;
    a.ldb = p.ld_w;
    a.M = p.rows;
    a.N = p.hidden;
    a.K = p.in;
    a.dt = dt_code(p.dtype);
    a.a_kc = 1;
    a.b_kc = oi;
    a.a_dma = operand_dma(p.x, p.ld_x, p.in, true, es);
    a.b_dma = operand_dma(p.w_gate, p.ld_w, oi ? p.in : p.hidden, oi, es) && aligned(p.w_up, 16);
    a.out = p.h;
    a.ld_out = p.ld_h;
    a.out_dt = a.dt;
    a.out_vec = rows_vec(p.h, p.ld_h, p.dtype);
    a.bias = p.bias_gate;
    a.bias2 = p.bias_up;
    a.bias_dt = dt_code(p.bias_dtype);
    a.bias_vec = aligned(p.bias_gate, 16) && aligned(p.bias_up, 16);
    a.z = p.gate;
    a.z2 = p.up;
    a.ld_z = p.ld_z;
    a.z_vec = p.gate && pair_vec(p.gate, p.up, p.ld_z, p.dtype);
    a.z8 = act8_view(p.gate8);
    a.z8_2 = act8_view(p.up8);
    return run_gated(h, a, static_cast<hipStream_t>(stream));
}

muon_status gated_grad_hidden(muon_handle* handle, const muon_gated_grad_hidden_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_gated_grad_hidden_args& p = *args;
    ck.dtype(p.dtype, "dy");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.hidden, 1, kMaxCols, "hidden");
    ck.size(p.out, 1, kMaxCols, "out");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.activation >= MUON_GATE_SILU && p.activation <= MUON_GATE_RELU, "unknown activation %d", p.activation);
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || (p.dy && p.dgate && p.dup), "dy, dgate or dup is NULL");
    ck.need(p.rows == 0 || p.gate || p.gate8.codes, "gate and up (or gate8 and up8) are NULL");
    ck.need(p.w_down != nullptr, "w_down is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN;
    ck.matrix(p.dy, p.ld_dy, p.out, p.dtype, "dy");
    ck.matrix(p.w_down, p.ld_w, oi ? p.hidden : p.out, p.dtype, "w_down");
    check_pair(ck, p.gate, p.up, p.gate8, p.up8, p.ld_z, p.hidden, p.dtype);
    ck.matrix(p.dgate, p.ld_dz, p.hidden, p.dtype, "dgate");
    ck.matrix(p.dup, p.ld_dz, p.hidden, p.dtype, "dup");
    ck.matrix(p.h, p.ld_h, p.hidden, p.dtype, "h");
    ck.distinct({p.dgate, p.dup, p.h},
                {p.dy, p.w_down, p.gate, p.up, p.gate8.codes, p.gate8.exponents, p.up8.codes, p.up8.exponents});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    GatedArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_GATED_DH;
    a.pair = PAIR_NONE;
    a.gate_act = p.activation;
    a.a = p.dy;
    a.b = p.w_down;
    a.lda = p.ld_dy;
    a.ldb = p.ld_w;
    a.M = p.rows;
    a.N = p.hidden;
    a.K = p.out;
    a.dt = dt_code(p.dtype);
    a.a_kc = 1;
    a.b_kc = !oi;
    a.a_dma = operand_dma(p.dy, p.ld_dy, p.out, true, es);
    a.b_dma = operand_dma(p.w_down, p.ld_w, oi ? p.hidden : p.out, !oi, es);
    a.out = p.dgate;
    a.out2 = p.dup;
    a.ld_out = p.ld_dz;
    a.out_dt = a.dt;
    a.out_vec = pair_vec(p.dgate, p.dup, p.ld_dz, p.dtype);
    a.z = const_cast<void*>(p.gate);
    a.z2 = const_cast<void*>(p.up);
    a.ld_z = p.ld_z;
    a.z_vec = p.gate && pair_vec(p.gate, p.up, p.ld_z, p.dtype);
    a.z8 = act8_view(p.gate8);
    a.z8_2 = act8_view(p.up8);
    a.act_out = p.h;
    a.ld_act = p.ld_h;
    a.act_vec = p.h && rows_vec(p.h, p.ld_h, p.dtype);
    return run_gated(h, a, static_cast<hipStream_t>(stream));
}

muon_status gated_grad_input(muon_handle* handle, const muon_gated_grad_input_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_gated_grad_input_args& p = *args;
    ck.dtype(p.dtype, "dgate");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.in, 1, kMaxCols, "in");
    ck.size(p.hidden, 1, kMaxCols, "hidden");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || (p.dgate && p.dup && p.dx), "dgate, dup or dx is NULL");
    ck.need(p.w_gate && p.w_up, "w_gate or w_up is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN;
    ck.matrix(p.dgate, p.ld_dz, p.hidden, p.dtype, "dgate");
    ck.matrix(p.dup, p.ld_dz, p.hidden, p.dtype, "dup");
    ck.matrix(p.w_gate, p.ld_w, oi ? p.in : p.hidden, p.dtype, "w_gate");
    ck.matrix(p.w_up, p.ld_w, oi ? p.in : p.hidden, p.dtype, "w_up");
    ck.matrix(p.add, p.ld_add, p.in, p.dtype, "add");
    ck.matrix(p.dx, p.ld_dx, p.in, p.dtype, "dx");
    ck.need(!p.add || p.add != p.dx || p.ld_add == p.ld_dx, "add is dx with another leading dimension");
    ck.distinct({p.dx}, {p.dgate, p.dup, p.w_gate, p.w_up, p.add == p.dx ? nullptr : p.add});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    GatedArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_DX;
    a.pair = PAIR_K;
    a.a = p.dgate;
    a.a2 = p.dup;
    a.b = p.w_gate;
    a.b2 = p.w_up;
    a.lda = p.ld_dz;
    a.ldb = p.ld_w;
    a.M = p.rows;
    a.N = p.in;
    a.K = p.hidden;
    a.dt = dt_code(p.dtype);
    a.a_kc = 1;
    a.b_kc = !oi;
    a.a_dma = operand_dma(p.dgate, p.ld_dz, p.hidden, true, es) && aligned(p.dup, 16);
    a.b_dma = operand_dma(p.w_gate, p.ld_w, oi ? p.in : p.hidden, !oi, es) && aligned(p.w_up, 16);
    a.out = p.dx;
    a.ld_out = p.ld_dx;
    a.out_dt = a.dt;
    a.out_vec = rows_vec(p.dx, p.ld_dx, p.dtype);
    a.add = p.add;
    a.ld_add = p.ld_add;
    a.add_vec = p.add && rows_vec(p.add, p.ld_add, p.dtype);
    return run_gated(h, a, static_cast<hipStream_t>(stream));
}

muon_status gated_grad_weight(muon_handle* handle, const muon_gated_grad_weight_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_gated_grad_weight_args& p = *args;
    ck.dtype(p.dtype, "dgate");
    ck.dtype(p.dw_dtype, "dw_gate");
    if (p.db_gate || p.db_up) ck.dtype(p.db_dtype, "db_gate");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.in, 1, kMaxCols, "in");
    ck.size(p.hidden, 1, kMaxCols, "hidden");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.accumulate == 0 || p.accumulate == 1, "accumulate must be 0 or 1, got %d", p.accumulate);
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || ((p.x || p.x8.codes) && p.dgate && p.dup), "x (or x8), dgate or dup is NULL");
    ck.need(!(p.x && p.x8.codes), "both x and x8");
    ck.need(p.dw_gate && p.dw_up, "dw_gate or dw_up is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN;
    ck.matrix(p.x, p.ld_x, p.in, p.dtype, "x");
    ck.matrix(p.dgate, p.ld_dz, p.hidden, p.dtype, "dgate");
    ck.matrix(p.dup, p.ld_dz, p.hidden, p.dtype, "dup");
    ck.matrix(p.dw_gate, p.ld_dw, oi ? p.in : p.hidden, p.dw_dtype, "dw_gate");
    ck.matrix(p.dw_up, p.ld_dw, oi ? p.in : p.hidden, p.dw_dtype, "dw_up");
    ck.vector(p.db_gate, p.db_dtype, "db_gate");
    ck.vector(p.db_up, p.db_dtype, "db_up");
    ck.act8(p.x8, p.in, "x8");
    ck.distinct({p.dw_gate, p.dw_up, p.db_gate, p.db_up}, {p.x, p.x8.codes, p.x8.exponents, p.dgate, p.dup});
    if (ck.st != MUON_OK) return ck.st;
    GatedArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_DW;
    a.pair = PAIR_OUT;
    a.M = p.in;
    a.N = p.hidden;
    a.K = p.rows;
    a.dt = dt_code(p.dtype);
    const bool x8 = p.x == nullptr && p.x8.codes != nullptr;
    a.a = x8 ? static_cast<const void*>(p.x8.codes) : p.x;
    a.lda = x8 ? p.x8.ld_codes : p.ld_x;
    a.a_exps = x8 ? p.x8.exponents : nullptr;
    a.lda_exps = x8 ? p.x8.ld_exponents : 0;
    a.a8_vec = x8 && act8_view(p.x8).vec;
    a.b = p.dgate;
    a.b2 = p.dup;
    a.ldb = p.ld_dz;
    a.a_dma = !x8 && operand_dma(p.x, p.ld_x, p.in, false, es);
    a.b_dma = operand_dma(p.dgate, p.ld_dz, p.hidden, false, es) && aligned(p.dup, 16);
    a.out = p.dw_gate;
    a.out2 = p.dw_up;
    a.ld_out = p.ld_dw;
    a.out_trans = oi;
    a.out_dt = dt_code(p.dw_dtype);
    a.out_vec = pair_vec(p.dw_gate, p.dw_up, p.ld_dw, p.dw_dtype);
    a.accumulate = p.accumulate;
    a.db = p.db_gate;
    a.db2 = p.db_up;
    a.db_dt = dt_code(p.db_dtype);
    if (p.rows == 0) {   // nothing to load: empty operands need no re-laying
        a.a_exps = nullptr;
        a.a_dma = a.b_dma = 1;
    }
    return run_gated(h, a, static_cast<hipStream_t>(stream));
}

void check_drop(Check& ck, const muon_dropout_mask& d) {
    ck.need(d.p >= 0.f && d.p <= 1.f, "the probability of dropping must lie in 0..1");
    ck.need(d.reserved == 0, "reserved field of the mask must be 0");
    ck.need(aligned(d.step, 8), "step: address not aligned to its elements");
}
DropMask drop_mask(const muon_dropout_mask& d) {
    DropMask m;
    m.seed = d.seed;
    m.offset = d.offset;
    m.step = d.step;
    m.cut = uint32_t(std::nearbyint(double(d.p) * 65536.0));
    m.scale = m.cut < 65536 ? float(65536.0 / double(65536 - m.cut)) : 0.f;
    return m;
}

muon_status dropout(muon_handle* handle, const muon_dropout_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_dropout_args& p = *args;
    ck.dtype(p.dtype, "x");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.cols, 1, kMaxCols, "cols");
    ck.need(p.reserved == 0, "reserved field must be 0");
    check_drop(ck, p.drop);
    ck.need(p.rows == 0 || (p.x && p.y), "x or y is NULL");
    ck.matrix(p.x, p.ld_x, p.cols, p.dtype, "x");
    ck.matrix(p.add, p.ld_add, p.cols, p.dtype, "add");
    ck.matrix(p.y, p.ld_y, p.cols, p.dtype, "y");
    ck.need(!p.x || p.x != p.y || p.ld_x == p.ld_y, "x is y with another leading dimension");
    ck.need(!p.add || p.add != p.y || p.ld_add == p.ld_y, "add is y with another leading dimension");
    ck.distinct({p.y}, {p.drop.step});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    DropoutArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = p.x;
    a.add = p.add;
    a.y = p.y;
    a.drop = drop_mask(p.drop);
    a.rows = p.rows;
    a.ld_x = p.ld_x;
    a.ld_add = p.ld_add;
    a.ld_y = p.ld_y;
    a.cols = int32_t(p.cols);
    a.dt = dt_code(p.dtype);
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    const hipError_t e = launch_dropout(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(h, e, "dropout launch");
    return MUON_OK;
}

bool known_norm(int32_t n) { return n >= MUON_NORM_NONE && n <= MUON_NORM_LAYER; }

// What both directions of a junction ask for.
template <class P>
void check_junction(Check& ck, const P& p) {
    ck.dtype(p.stream_dtype, "stream");
    ck.dtype(p.dtype, "block");
    ck.dtype(p.param_dtype, "parameters");
    if (ck.st == MUON_OK && p.stream_dtype == MUON_BF16 && p.dtype == MUON_F32)
        ck.st = fail(ck.h, MUON_ERR_DTYPE, "a bf16 stream between float32 blocks");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.cols, 1, kMaxCols, "cols");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(known_norm(p.post_norm) && known_norm(p.pre_norm), "unknown norm %d or %d", p.post_norm, p.pre_norm);
    ck.need(std::isfinite(p.residual_scale) && std::isfinite(p.branch_scale), "scales must be finite");
    check_drop(ck, p.drop);
    ck.need(p.post_norm || (!p.post_gain && !p.post_bias), "a gain or bias without post_norm");
    ck.need(p.pre_norm || !p.pre_gain, "a gain without pre_norm");
    ck.need(p.post_norm == MUON_NORM_LAYER || !p.post_bias, "post_bias without a layer norm");
    for (const void* v : {p.post_gain, p.post_bias, p.gate, p.pre_gain}) ck.vector(v, p.param_dtype, "a parameter");
    for (const float* v : {p.post_mean, p.post_rstd, p.pre_mean, p.pre_rstd}) ck.vector(v, MUON_F32, "a statistic");
}

muon_status blocknorm_forward(muon_handle* handle, const muon_blocknorm_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_blocknorm_args& p = *args;
    check_junction(ck, p);
    const bool empty = p.rows == 0;
    ck.need(std::isfinite(p.post_eps) && p.post_eps >= 0.f && std::isfinite(p.pre_eps) && p.pre_eps >= 0.f,
            "eps must be finite and >= 0");
    ck.need(p.pre_norm == MUON_NORM_LAYER || !p.pre_bias, "pre_bias without a layer norm");
    ck.vector(p.pre_bias, p.param_dtype, "a parameter");
    ck.need(empty || p.x, "x is NULL");
    ck.need(empty || !p.branch || p.s, "s is NULL beside a branch");
    ck.need(empty || p.branch || (!p.s && p.post_norm == MUON_NORM_NONE && !p.gate && p.residual_scale == 1.f && p.drop.p == 0.f),
            "s, a post norm, gate, residual_scale or dropout without a branch");
    ck.need(empty || p.branch || p.pre_norm, "neither a branch nor pre_norm");
    ck.need(empty || (p.y != nullptr) == (p.pre_norm != MUON_NORM_NONE), "y goes with pre_norm");
    ck.need(p.pre_norm || !p.y8.codes, "y8 without pre_norm");
    ck.need((p.post_norm || !p.post_rstd) && (p.pre_norm || !p.pre_rstd) &&
                (p.post_norm == MUON_NORM_LAYER || !p.post_mean) && (p.pre_norm == MUON_NORM_LAYER || !p.pre_mean),
            "a statistic of no norm, or a mean without a layer norm");
    ck.matrix(p.x, p.ld_x, p.cols, p.stream_dtype, "x");
    ck.matrix(p.branch, p.ld_branch, p.cols, p.dtype, "branch");
    ck.matrix(p.s, p.ld_s, p.cols, p.stream_dtype, "s");
    ck.matrix(p.y, p.ld_y, p.cols, p.dtype, "y");
    ck.act8(p.y8, p.cols, "y8");
    ck.need(!p.s || p.s != p.x || p.ld_s == p.ld_x, "s is x with another leading dimension");
    ck.distinct({p.s, p.y, p.y8.codes, p.y8.exponents, p.post_mean, p.post_rstd, p.pre_mean, p.pre_rstd},
                {p.x == p.s ? nullptr : p.x, p.branch, p.post_gain, p.post_bias, p.gate, p.pre_gain, p.pre_bias, p.drop.step});
    if (ck.st != MUON_OK) return ck.st;
    if (empty) return MUON_OK;
    BlockNormArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = p.x;
    a.branch = p.branch;
    a.post_gain = p.post_gain;
    a.post_bias = p.post_bias;
    a.gate = p.gate;
    a.pre_gain = p.pre_gain;
    a.pre_bias = p.pre_bias;
    a.s = p.s;
    a.y = p.y;
    a.y8 = act8_view(p.y8);
    a.post_mean = p.post_mean;
    a.post_rstd = p.post_rstd;
    a.pre_mean = p.pre_mean;
    a.pre_rstd = p.pre_rstd;
    a.drop = drop_mask(p.drop);
    a.rows = p.rows;
    a.cols = int32_t(p.cols);
    a.ld_x = p.ld_x;
    a.ld_branch = p.ld_branch;
    a.ld_s = p.ld_s;
    a.ld_y = p.ld_y;
    a.alpha = p.residual_scale;
    a.beta = p.branch_scale;
    a.post_eps = p.post_eps;
    a.pre_eps = p.pre_eps;
    a.post = p.post_norm;
    a.pre = p.pre_norm;
    a.sdt = dt_code(p.stream_dtype);
    a.dt = dt_code(p.dtype);
    a.pdt = dt_code(p.param_dtype);
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    const hipError_t e = launch_blocknorm(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(h, e, "block norm launch");
    return MUON_OK;
}

muon_status blocknorm_backward(muon_handle* handle, const muon_blocknorm_grad_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_blocknorm_grad_args& p = *args;
    check_junction(ck, p);
    const bool empty = p.rows == 0;
    ck.need(p.accumulate == 0 || p.accumulate == 1, "accumulate must be 0 or 1, got %d", p.accumulate);
    ck.need(empty || p.dx, "dx is NULL");
    ck.need(empty || p.pre_norm || p.ds, "neither ds nor pre_norm");
    ck.need(empty || (p.dy != nullptr) == (p.pre_norm != MUON_NORM_NONE), "dy goes with pre_norm");
    ck.need(empty || !p.pre_norm || (p.s && p.pre_rstd && (p.pre_norm != MUON_NORM_LAYER || p.pre_mean)),
            "pre_norm without s or its statistics");
    ck.need(empty || !p.post_norm || (p.branch && p.post_rstd && (p.post_norm != MUON_NORM_LAYER || p.post_mean)),
            "post_norm without branch or its statistics");
    ck.need(empty || p.dbranch || (!p.branch && p.post_norm == MUON_NORM_NONE && !p.gate && p.drop.p == 0.f),
            "a branch, post norm, gate or dropout without dbranch");
    ck.need(p.post_gain || !p.dpost_gain, "dpost_gain without post_gain");
    ck.need(p.post_bias || !p.dpost_bias, "dpost_bias without post_bias");
    ck.need(p.gate || !p.dgate, "dgate without gate");
    ck.need(empty || p.branch || !p.dgate, "dgate without branch");
    ck.need(p.pre_gain || !p.dpre_gain, "dpre_gain without pre_gain");
    ck.need(p.pre_norm == MUON_NORM_LAYER || !p.dpre_bias, "dpre_bias without a layer norm");
    ck.matrix(p.dy, p.ld_dy, p.cols, p.dtype, "dy");
    ck.matrix(p.ds, p.ld_ds, p.cols, p.stream_dtype, "ds");
    ck.matrix(p.s, p.ld_s, p.cols, p.stream_dtype, "s");
    ck.matrix(p.branch, p.ld_branch, p.cols, p.dtype, "branch");
    ck.matrix(p.dx, p.ld_dx, p.cols, p.stream_dtype, "dx");
    ck.matrix(p.dbranch, p.ld_dbranch, p.cols, p.dtype, "dbranch");
    for (const void* v : {p.dpost_gain, p.dpost_bias, p.dgate, p.dpre_gain, p.dpre_bias})
        ck.vector(v, p.param_dtype, "a parameter's gradient");
    ck.need(!p.ds || p.ds != p.dx || p.ld_ds == p.ld_dx, "ds is dx with another leading dimension");
    ck.distinct({p.dx, p.dbranch, p.dpost_gain, p.dpost_bias, p.dgate, p.dpre_gain, p.dpre_bias},
                {p.dy, p.ds == p.dx ? nullptr : p.ds, p.s, p.branch, p.post_gain, p.post_bias, p.gate, p.pre_gain,
                 p.post_mean, p.post_rstd, p.pre_mean, p.pre_rstd, p.drop.step});
    if (ck.st != MUON_OK) return ck.st;
    BlockNormGradArgs a;
    std::memset(&a, 0, sizeof a);
    a.dy = p.dy;
    a.ds = p.ds;
    a.s = p.s;
    a.branch = p.branch;
    a.post_gain = p.post_gain;
    a.post_bias = p.post_bias;
    a.gate = p.gate;
    a.pre_gain = p.pre_gain;
    a.post_mean = p.post_mean;
    a.post_rstd = p.post_rstd;
    a.pre_mean = p.pre_mean;
    a.pre_rstd = p.pre_rstd;
    a.dx = p.dx;
    a.dbranch = p.dbranch;
    a.dpost_gain = p.dpost_gain;
    a.dpost_bias = p.dpost_bias;
    a.dgate = p.dgate;
    a.dpre_gain = p.dpre_gain;
    a.dpre_bias = p.dpre_bias;
    a.drop = drop_mask(p.drop);
    a.rows = p.rows;
    a.cols = int32_t(p.cols);
    a.ld_dy = p.ld_dy;
    a.ld_ds = p.ld_ds;
    a.ld_s = p.ld_s;
    a.ld_branch = p.ld_branch;
    a.ld_dx = p.ld_dx;
    a.ld_dbranch = p.ld_dbranch;
    a.alpha = p.residual_scale;
    a.beta = p.branch_scale;
    a.post = p.post_norm;
    a.pre = p.pre_norm;
    a.sdt = dt_code(p.stream_dtype);
    a.dt = dt_code(p.dtype);
    a.pdt = dt_code(p.param_dtype);
    a.accumulate = p.accumulate;
    const bool want[4] = {p.dpre_gain != nullptr, p.dpre_bias != nullptr, p.dpost_gain || p.dgate,
                          p.dpost_bias || (p.dgate && p.post_bias)};
    for (int i = 0; i < 4; ++i) a.at[i] = want[i] ? a.sums++ : -1;
    a.parts = blocknorm_parts(a);
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    void* ws = nullptr;
    const muon_status st = workspace(h, size_t(a.sums) * size_t(a.parts) * size_t(p.cols) * 4, static_cast<hipStream_t>(stream), &ws);
    if (st != MUON_OK) return st;
    a.partial = static_cast<float*>(ws);
    const hipError_t e = launch_blocknorm_grad(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(h, e, "block norm gradient launch");
    return MUON_OK;
}

}  // namespace

extern "C" {

muon_status muon_gated_forward(muon_handle* h, const muon_gated_args* args, void* stream) {
    return guarded([&] { return gated_forward(h, args, stream); });
}
muon_status muon_gated_grad_hidden(muon_handle* h, const muon_gated_grad_hidden_args* args, void* stream) {
    return guarded([&] { return gated_grad_hidden(h, args, stream); });
}
muon_status muon_gated_grad_input(muon_handle* h, const muon_gated_grad_input_args* args, void* stream) {
    return guarded([&] { return gated_grad_input(h, args, stream); });
}
muon_status muon_gated_grad_weight(muon_handle* h, const muon_gated_grad_weight_args* args, void* stream) {
    return guarded([&] { return gated_grad_weight(h, args, stream); });
}
muon_status muon_dropout(muon_handle* h, const muon_dropout_args* args, void* stream) {
    return guarded([&] { return dropout(h, args, stream); });
}
muon_status muon_blocknorm_forward(muon_handle* h, const muon_blocknorm_args* args, void* stream) {
    return guarded([&] { return blocknorm_forward(h, args, stream); });
}
muon_status muon_blocknorm_backward(muon_handle* h, const muon_blocknorm_grad_args* args, void* stream) {
    return guarded([&] { return blocknorm_backward(h, args, stream); });
}

}  // extern "C"
