// Host side of the layer operators: argument validation, workspaces and
// launches.  Each call validates everything before it enqueues anything.

#include "layer_host.hpp"

using namespace muon;

static_assert(MUON_ACT8_GROUP == kAct8Group, "the ABI's group size");
static_assert(int(MUON_ACT_GELU) == int(ACT_GELU) && int(MUON_ACT_RELU_SQ) == int(ACT_RELU_SQ), "activation codes");

namespace {

muon_status run_linear(HandleBase* h, LinArgs& a, hipStream_t stream) {
    const int64_t tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128);
    if (tiles > kMaxTiles128)
        return fail(h, MUON_ERR_INVALID_ARG, "more than %lld output tiles of 128 x 128", (long long)kMaxTiles128);
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    const LinPlan p = plan_linear(a);
    a.splits = p.splits;
    a.tile = p.tile;
    a.deep = p.deep;
    void* ws = nullptr;
    auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
    const size_t at[4] = {0, up(p.partial_bytes), up(p.partial_bytes) + up(p.db_bytes),
                          up(p.partial_bytes) + up(p.db_bytes) + up(p.a_bytes)};
    const muon_status st = workspace(h, at[3] + p.b_bytes, stream, &ws);
    if (st != MUON_OK) return st;
    char* base = static_cast<char*>(ws);
    if (p.partial_bytes) a.partial = reinterpret_cast<float*>(base);
    if (p.db_bytes) a.db_partial = reinterpret_cast<float*>(base + at[1]);
    if (p.a_bytes) a.a_ws = base + at[2];
    if (p.b_bytes) a.b_ws = base + at[3];
    a.a_ld = p.a_ld;
    a.b_ld = p.b_ld;
    const hipError_t e = launch_linear(a, stream);
    if (e != hipSuccess) return hip_fail(h, e, "linear launch");
    return MUON_OK;
}

}  // namespace

namespace {

muon_status layernorm_forward(muon_handle* handle, const muon_layernorm_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_layernorm_args& p = *args;
    ck.dtype(p.dtype, "x");
    ck.dtype(p.param_dtype, "gain");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.cols, 1, kMaxCols, "cols");
    ck.need(norm_rows_fit(p.rows, p.cols), "too many rows of %lld columns", (long long)p.cols);
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(std::isfinite(p.eps) && p.eps >= 0.f, "eps must be finite and >= 0");
    ck.need(p.rows == 0 || (p.x && p.y), "x or y is NULL");
    ck.need(p.gain != nullptr, "gain is NULL");
    ck.matrix(p.x, p.ld_x, p.cols, p.dtype, "x");
    ck.matrix(p.y, p.ld_y, p.cols, p.dtype, "y");
    ck.vector(p.gain, p.param_dtype, "gain");
    ck.vector(p.bias, p.param_dtype, "bias");
    ck.vector(p.mean, MUON_F32, "mean");
    ck.vector(p.rstd, MUON_F32, "rstd");
    ck.act8(p.y8, p.cols, "y8");
    ck.distinct({p.y, p.mean, p.rstd, p.y8.codes, p.y8.exponents}, {p.x, p.gain, p.bias});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    NormArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = p.x;
    a.y = p.y;
    a.gain = p.gain;
    a.bias = p.bias;
    a.mean = p.mean;
    a.rstd = p.rstd;
    a.y8 = act8_view(p.y8);
    a.rows = p.rows;
    a.cols = int32_t(p.cols);
    a.ld_x = p.ld_x;
    a.ld_y = p.ld_y;
    a.dt = dt_code(p.dtype);
    a.pdt = dt_code(p.param_dtype);
    const int v = 16 / esize(p.dtype);
    a.vec = p.cols % v == 0 && rows_vec(p.x, p.ld_x, p.dtype) && rows_vec(p.y, p.ld_y, p.dtype);
    a.pvec = aligned(p.gain, 16) && aligned(p.bias, 16);
    a.eps = p.eps;
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    const hipError_t e = launch_norm(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(h, e, "layer norm launch");
    return MUON_OK;
}

muon_status layernorm_backward(muon_handle* handle, const muon_layernorm_grad_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_layernorm_grad_args& p = *args;
    ck.dtype(p.dtype, "x");
    ck.dtype(p.param_dtype, "gain");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.cols, 1, kMaxCols, "cols");
    ck.need(norm_rows_fit(p.rows, p.cols), "too many rows of %lld columns", (long long)p.cols);
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.accumulate == 0 || p.accumulate == 1, "accumulate must be 0 or 1, got %d", p.accumulate);
    ck.need(p.rows == 0 || (p.dy && p.x && p.mean && p.rstd && p.dx), "dy, x, mean, rstd or dx is NULL");
    ck.need(p.gain && p.dgain, "gain or dgain is NULL");
    ck.matrix(p.dy, p.ld_dy, p.cols, p.dtype, "dy");
    ck.matrix(p.x, p.ld_x, p.cols, p.dtype, "x");
    ck.matrix(p.add, p.ld_add, p.cols, p.dtype, "add");
    ck.matrix(p.dx, p.ld_dx, p.cols, p.dtype, "dx");
    ck.vector(p.gain, p.param_dtype, "gain");
    ck.vector(p.dgain, p.param_dtype, "dgain");
    ck.vector(p.dbias, p.param_dtype, "dbias");
    ck.vector(p.mean, MUON_F32, "mean");
    ck.vector(p.rstd, MUON_F32, "rstd");
    ck.need(!p.add || p.add != p.dx || p.ld_add == p.ld_dx, "add is dx with another leading dimension");
    ck.distinct({p.dx, p.dgain, p.dbias}, {p.dy, p.x, p.gain, p.mean, p.rstd, p.add == p.dx ? nullptr : p.add});
    if (ck.st != MUON_OK) return ck.st;
    NormGradArgs a;
    std::memset(&a, 0, sizeof a);
    a.dy = p.dy;
    a.x = p.x;
    a.gain = p.gain;
    a.mean = p.mean;
    a.rstd = p.rstd;
    a.add = p.add;
    a.dx = p.dx;
    a.dgain = p.dgain;
    a.dbias = p.dbias;
    a.rows = p.rows;
    a.cols = int32_t(p.cols);
    a.ld_dy = p.ld_dy;
    a.ld_x = p.ld_x;
    a.ld_add = p.ld_add;
    a.ld_dx = p.ld_dx;
    a.dt = dt_code(p.dtype);
    a.pdt = dt_code(p.param_dtype);
    const int v = 16 / esize(p.dtype);
    a.vec = p.cols % v == 0 && rows_vec(p.x, p.ld_x, p.dtype) && rows_vec(p.dy, p.ld_dy, p.dtype) &&
            rows_vec(p.dx, p.ld_dx, p.dtype) && (!p.add || rows_vec(p.add, p.ld_add, p.dtype));
    a.pvec = aligned(p.gain, 16);
    a.accumulate = p.accumulate;
    a.parts = norm_grad_parts(p.rows, int(p.cols));
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    void* ws = nullptr;
    const muon_status st = workspace(h, size_t(2) * size_t(a.parts) * size_t(p.cols) * 4, static_cast<hipStream_t>(stream), &ws);
    if (st != MUON_OK) return st;
    a.partial = static_cast<float*>(ws);
    const hipError_t e = launch_norm_grad(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(h, e, "layer norm gradient launch");
    return MUON_OK;
}

muon_status linear_forward(muon_handle* handle, const muon_linear_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_linear_args& p = *args;
    ck.dtype(p.dtype, "x");
    if (p.bias) ck.dtype(p.bias_dtype, "bias");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.in, 1, kMaxCols, "in");
    ck.size(p.out, 1, kMaxCols, "out");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.activation >= MUON_ACT_NONE && p.activation <= MUON_ACT_RELU_SQ, "unknown activation %d", p.activation);
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || (p.x && p.y), "x or y is NULL");
    ck.need(p.w != nullptr, "w is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN;
    ck.matrix(p.x, p.ld_x, p.in, p.dtype, "x");
    ck.matrix(p.w, p.ld_w, oi ? p.in : p.out, p.dtype, "w");
    ck.matrix(p.residual, p.ld_residual, p.out, p.dtype, "residual");
    ck.matrix(p.y, p.ld_y, p.out, p.dtype, "y");
    ck.matrix(p.z, p.ld_z, p.out, p.dtype, "z");
    ck.vector(p.bias, p.bias_dtype, "bias");
    ck.act8(p.z8, p.out, "z8");
    ck.need(!(p.z && p.z8.codes), "both z and z8");
    ck.need(!p.residual || p.residual != p.y || p.ld_residual == p.ld_y, "residual is y with another leading dimension");
    ck.distinct({p.y, p.z, p.z8.codes, p.z8.exponents},
                {p.x, p.w, p.bias, p.residual == p.y ? nullptr : p.residual});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    LinArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_FWD;
    a.act = p.activation;
    a.a = p.x;
    a.b = p.w;
    a.lda = p.ld_x;
    a.ldb = p.ld_w;
    a.M = p.rows;
    a.N = p.out;
    a.K = p.in;
    a.dt = dt_code(p.dtype);
    a.a_kc = 1;
    a.b_kc = oi;
    a.a_dma = operand_dma(p.x, p.ld_x, p.in, true, es);
    a.b_dma = operand_dma(p.w, p.ld_w, oi ? p.in : p.out, oi, es);
    a.out = p.y;
    a.ld_out = p.ld_y;
    a.out_dt = a.dt;
    a.out_vec = rows_vec(p.y, p.ld_y, p.dtype);
    a.bias = p.bias;
    a.bias_dt = dt_code(p.bias_dtype);
    a.bias_vec = aligned(p.bias, 16);
    a.add = p.residual;
    a.ld_add = p.ld_residual;
    a.add_vec = p.residual && rows_vec(p.residual, p.ld_residual, p.dtype);
    a.z = p.z;
    a.ld_z = p.ld_z;
    a.z_vec = p.z && rows_vec(p.z, p.ld_z, p.dtype);
    a.z8 = act8_view(p.z8);
    return run_linear(h, a, static_cast<hipStream_t>(stream));
}

muon_status linear_grad_input(muon_handle* handle, const muon_linear_grad_input_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_linear_grad_input_args& p = *args;
    ck.dtype(p.dtype, "dy");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.in, 1, kMaxCols, "in");
    ck.size(p.out, 1, kMaxCols, "out");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.activation >= MUON_ACT_NONE && p.activation <= MUON_ACT_RELU_SQ, "unknown activation %d", p.activation);
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || (p.dy && p.dx), "dy or dx is NULL");
    ck.need(p.w != nullptr, "w is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN, has_z = p.z || p.z8.codes;
    ck.matrix(p.dy, p.ld_dy, p.out, p.dtype, "dy");
    ck.matrix(p.w, p.ld_w, oi ? p.in : p.out, p.dtype, "w");
    ck.matrix(p.z, p.ld_z, p.in, p.dtype, "z");
    ck.matrix(p.add, p.ld_add, p.in, p.dtype, "add");
    ck.matrix(p.dx, p.ld_dx, p.in, p.dtype, "dx");
    ck.matrix(p.act_out, p.ld_act_out, p.in, p.dtype, "act_out");
    ck.act8(p.z8, p.in, "z8");
    ck.need(!(p.z && p.z8.codes), "both z and z8");
    const bool z_known = has_z || p.rows == 0;   // an empty tensor's address is null
    ck.need(z_known || !p.act_out, "act_out without z or z8");
    ck.need(z_known || p.activation == MUON_ACT_NONE, "an activation without z or z8");
    ck.need(!p.add || p.add != p.dx || p.ld_add == p.ld_dx, "add is dx with another leading dimension");
    ck.distinct({p.dx, p.act_out},
                {p.dy, p.w, p.z, p.z8.codes, p.z8.exponents, p.add == p.dx ? nullptr : p.add});
    if (ck.st != MUON_OK) return ck.st;
    if (p.rows == 0) return MUON_OK;
    LinArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_DX;
    a.act = p.activation;
    a.a = p.dy;
    a.b = p.w;
    a.lda = p.ld_dy;
    a.ldb = p.ld_w;
    a.M = p.rows;
    a.N = p.in;
    a.K = p.out;
    a.dt = dt_code(p.dtype);
    a.a_kc = 1;
    a.b_kc = !oi;
    a.a_dma = operand_dma(p.dy, p.ld_dy, p.out, true, es);
    a.b_dma = operand_dma(p.w, p.ld_w, oi ? p.in : p.out, !oi, es);
    a.out = p.dx;
    a.ld_out = p.ld_dx;
    a.out_dt = a.dt;
    a.out_vec = rows_vec(p.dx, p.ld_dx, p.dtype);
    a.add = p.add;
    a.ld_add = p.ld_add;
    a.add_vec = p.add && rows_vec(p.add, p.ld_add, p.dtype);
    a.z = const_cast<void*>(p.z);
    a.ld_z = p.ld_z;
    a.z_vec = p.z && rows_vec(p.z, p.ld_z, p.dtype);
    a.z8 = act8_view(p.z8);
    a.act_out = p.act_out;
    a.ld_act = p.ld_act_out;
    a.act_vec = p.act_out && rows_vec(p.act_out, p.ld_act_out, p.dtype);
    // dx and act_out together past what the L2s hold (32 MiB): the lines of one
    // are sent out as they are written, not at the kernel's end (4001 x 1024,
    // weight 4096 x 1024, 2 x 31 MiB written: 58.1 -> 47.4 us; both streamed
    // 45.4, but the products that read dx next lose more than that).
    a.act_stream = p.act_out && 2 * p.rows * p.in * es > (32ll << 20);
    return run_linear(h, a, static_cast<hipStream_t>(stream));
}

muon_status linear_grad_weight(muon_handle* handle, const muon_linear_grad_weight_args* args, void* stream) {
    LAYER_ENTER(handle, args);
    const muon_linear_grad_weight_args& p = *args;
    ck.dtype(p.dtype, "dy");
    ck.dtype(p.dw_dtype, "dw");
    if (p.db) ck.dtype(p.db_dtype, "db");
    ck.size(p.rows, 0, kMaxRows, "rows");
    ck.size(p.in, 1, kMaxCols, "in");
    ck.size(p.out, 1, kMaxCols, "out");
    ck.need(p.reserved == 0, "reserved field must be 0");
    ck.need(p.accumulate == 0 || p.accumulate == 1, "accumulate must be 0 or 1, got %d", p.accumulate);
    ck.need(p.w_layout == MUON_W_IN_OUT || p.w_layout == MUON_W_OUT_IN, "unknown weight layout %d", p.w_layout);
    ck.need(p.rows == 0 || ((p.x || p.x8.codes) && p.dy), "x (or x8) or dy is NULL");
    ck.need(!(p.x && p.x8.codes), "both x and x8");
    ck.need(p.dw != nullptr, "dw is NULL");
    const bool oi = p.w_layout == MUON_W_OUT_IN;
    ck.matrix(p.x, p.ld_x, p.in, p.dtype, "x");
    ck.matrix(p.dy, p.ld_dy, p.out, p.dtype, "dy");
    ck.matrix(p.dw, p.ld_dw, oi ? p.in : p.out, p.dw_dtype, "dw");
    ck.vector(p.db, p.db_dtype, "db");
    ck.act8(p.x8, p.in, "x8");
    ck.distinct({p.dw, p.db}, {p.x, p.x8.codes, p.x8.exponents, p.dy});
    if (ck.st != MUON_OK) return ck.st;
    LinArgs a;
    std::memset(&a, 0, sizeof a);
    const int es = esize(p.dtype);
    a.kind = LIN_DW;
    a.M = p.in;
    a.N = p.out;
    a.K = p.rows;
    a.dt = dt_code(p.dtype);
    const bool x8 = p.x == nullptr && p.x8.codes != nullptr;
    a.a = x8 ? static_cast<const void*>(p.x8.codes) : p.x;
    a.lda = x8 ? p.x8.ld_codes : p.ld_x;
    a.a_exps = x8 ? p.x8.exponents : nullptr;
    a.lda_exps = x8 ? p.x8.ld_exponents : 0;
    a.a8_vec = x8 && act8_view(p.x8).vec;
    a.b = p.dy;
    a.ldb = p.ld_dy;
    a.a_dma = !x8 && operand_dma(p.x, p.ld_x, p.in, false, es);
    a.b_dma = operand_dma(p.dy, p.ld_dy, p.out, false, es);
    a.out = p.dw;
    a.ld_out = p.ld_dw;
    a.out_trans = oi;
    a.out_dt = dt_code(p.dw_dtype);
    a.out_vec = rows_vec(p.dw, p.ld_dw, p.dw_dtype);
    a.accumulate = p.accumulate;
    a.db = p.db;
    a.db_dt = dt_code(p.db_dtype);
    return run_linear(h, a, static_cast<hipStream_t>(stream));
}

muon_status run_act8(HandleBase* h, Act8Args& a, const muon_act8& q, const void* m, int64_t cols, int32_t dtype,
                     bool encode, hipStream_t stream) {
    a.q = act8_view(q);
    a.cols = int32_t(cols);
    a.dt = dt_code(dtype);
    a.vec = a.q.vec && rows_vec(m, a.ld, dtype);
    DeviceGuard g(h->device);
    if (!g.ok) return fail(h, MUON_ERR_NO_DEVICE, "cannot select device %d", h->device);
    const hipError_t e = encode ? launch_act8_encode(a, stream) : launch_act8_decode(a, stream);
    if (e != hipSuccess) return hip_fail(h, e, "checkpoint launch");
    return MUON_OK;
}

muon_status act_encode(muon_handle* handle, const void* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t dtype,
                            const muon_act8* q, void* stream) {
    LAYER_ENTER(handle, q);
    ck.dtype(dtype, "x");
    ck.size(rows, 0, kMaxRows, "rows");
    ck.size(cols, 1, kMaxCols, "cols");
    ck.need(rows == 0 || (x && q->codes), "x or the codes are NULL");
    ck.matrix(x, ld_x, cols, dtype, "x");
    ck.act8(*q, cols, "q");
    ck.distinct({q->codes, q->exponents}, {x});
    if (ck.st != MUON_OK) return ck.st;
    if (rows == 0) return MUON_OK;
    Act8Args a;
    std::memset(&a, 0, sizeof a);
    a.x = x;
    a.rows = rows;
    a.ld = ld_x;
    return run_act8(h, a, *q, x, cols, dtype, true, static_cast<hipStream_t>(stream));
}

muon_status act_decode(muon_handle* handle, const muon_act8* q, void* y, int64_t rows, int64_t cols, int64_t ld_y,
                            int32_t dtype, void* stream) {
    LAYER_ENTER(handle, q);
    ck.dtype(dtype, "y");
    ck.size(rows, 0, kMaxRows, "rows");
    ck.size(cols, 1, kMaxCols, "cols");
    ck.need(rows == 0 || (y && q->codes), "y or the codes are NULL");
    ck.matrix(y, ld_y, cols, dtype, "y");
    ck.act8(*q, cols, "q");
    ck.distinct({y}, {q->codes, q->exponents});
    if (ck.st != MUON_OK) return ck.st;
    if (rows == 0) return MUON_OK;
    Act8Args a;
    std::memset(&a, 0, sizeof a);
    a.y = y;
    a.rows = rows;
    a.ld = ld_y;
    return run_act8(h, a, *q, y, cols, dtype, false, static_cast<hipStream_t>(stream));
}

}  // namespace

extern "C" {

muon_status muon_layernorm_forward(muon_handle* h, const muon_layernorm_args* args, void* stream) {
    return guarded([&] { return layernorm_forward(h, args, stream); });
}
muon_status muon_layernorm_backward(muon_handle* h, const muon_layernorm_grad_args* args, void* stream) {
    return guarded([&] { return layernorm_backward(h, args, stream); });
}
muon_status muon_linear_forward(muon_handle* h, const muon_linear_args* args, void* stream) {
    return guarded([&] { return linear_forward(h, args, stream); });
}
muon_status muon_linear_grad_input(muon_handle* h, const muon_linear_grad_input_args* args, void* stream) {
    return guarded([&] { return linear_grad_input(h, args, stream); });
}
muon_status muon_linear_grad_weight(muon_handle* h, const muon_linear_grad_weight_args* args, void* stream) {
    return guarded([&] { return linear_grad_weight(h, args, stream); });
}
muon_status muon_act_encode(muon_handle* h, const void* x, int64_t rows, int64_t cols, int64_t ld_x, int32_t dtype,
                            const muon_act8* q, void* stream) {
    return guarded([&] { return act_encode(h, x, rows, cols, ld_x, dtype, q, stream); });
}
muon_status muon_act_decode(muon_handle* h, const muon_act8* q, void* y, int64_t rows, int64_t cols, int64_t ld_y,
                            int32_t dtype, void* stream) {
    return guarded([&] { return act_decode(h, q, y, rows, cols, ld_y, dtype, stream); });
}

}  // extern "C"
