// Test infrastructure: runs the block operators of the library, built against the
// CPU stand-in of HIP (tests/emu_layers), on exactly sized host buffers, so
// AddressSanitizer reports any access outside them.  Usage:
//   emu_blocks_driver OP ROWS A B DTYPE FLAGS PAD SHIFT | emu_blocks_driver refuse
// OP gated (A, B = in, hidden), norm or drop (A = cols); DTYPE 0 bf16, 1 float32,
// 2 a float32 stream between bf16 blocks (norm); FLAGS bit 0 weight layout out x
// in, bit 1 8-bit checkpoints, bit 2 without the optional arguments, bit 3 layer
// norms (else RMS), bit 4 without a branch, bit 5 in place; PAD extra elements per
// row, SHIFT elements by which every buffer starts past its allocation.  The bytes
// between rows are checked to keep their value.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>
#include <vector>

#include "muon.h"

emu_idx threadIdx, blockIdx;
dim3 gridDim, blockDim;
long emu_launches = 0;
int emu_verbose = 0;

struct Buf {
    char* alloc;
    char* p;
    long rows, cols, ld;
    int es;
    float* f() const { return reinterpret_cast<float*>(p); }
};
static std::vector<Buf> bufs;
static long g_pad, g_shift;

static Buf mat(long rows, long cols, int es) {
    Buf b{nullptr, nullptr, rows, cols, cols + g_pad, es};
    const long n = rows > 0 ? (rows - 1) * b.ld + cols + g_shift : g_shift;
    b.alloc = static_cast<char*>(std::malloc(n * es > 0 ? n * es : 1));
    b.p = b.alloc + g_shift * es;
    for (long r = 0; r < rows; ++r)
        for (long c = 0; c < (r + 1 < rows ? b.ld : cols); ++c) {
            char* q = b.p + (r * b.ld + c) * es;
            const float f = float((r * 7 + c * 3) % 13 - 6) * 0.25f;
            if (c >= cols) std::memset(q, 0x5A, es);
            else if (es == 4) std::memcpy(q, &f, 4);
            else if (es == 2) std::memcpy(q, reinterpret_cast<const char*>(&f) + 2, 2);
            else *q = char(120 + (r + c) % 8);   // as a code or as an exponent byte
        }
    bufs.push_back(b);
    return b;
}
static Buf vec(long n, int es) { return mat(1, n, es); }
static long damaged() {
    long bad = 0;
    for (const Buf& b : bufs)
        for (long r = 0; r + 1 < b.rows; ++r)
            for (long k = b.cols * b.es; k < b.ld * b.es; ++k) bad += b.p[r * b.ld * b.es + k] != 0x5A;
    return bad;
}
static muon_act8 act8(long rows, long cols) {
    const Buf q = mat(rows, cols, 1), e = mat(rows, (cols + 31) / 32, 1);
    return muon_act8{reinterpret_cast<int8_t*>(q.p), reinterpret_cast<uint8_t*>(e.p), q.ld, e.ld};
}

static muon_gated_args gated_args(long rows, long in, long hid, int es, int dt, bool oi) {
    muon_gated_args f{};
    const Buf x = mat(rows, in, es), h = mat(rows, hid, es), wg = oi ? mat(hid, in, es) : mat(in, hid, es),
              wu = oi ? mat(hid, in, es) : mat(in, hid, es);
    f.x = x.p, f.w_gate = wg.p, f.w_up = wu.p, f.h = h.p, f.rows = rows, f.in = in, f.hidden = hid;
    f.ld_x = x.ld, f.ld_w = wg.ld, f.ld_h = h.ld, f.dtype = f.bias_dtype = dt, f.w_layout = oi;
    return f;
}
static muon_gated_grad_hidden_args hidden_args(long rows, long hid, long out, int es, int dt, bool oi) {
    muon_gated_grad_hidden_args f{};
    const Buf dy = mat(rows, out, es), w = oi ? mat(out, hid, es) : mat(hid, out, es), dg = mat(rows, hid, es),
              du = mat(rows, hid, es), g = mat(rows, hid, es), u = mat(rows, hid, es);
    f.dy = dy.p, f.w_down = w.p, f.dgate = dg.p, f.dup = du.p, f.gate = g.p, f.up = u.p, f.rows = rows, f.hidden = hid;
    f.out = out, f.ld_dy = dy.ld, f.ld_w = w.ld, f.ld_z = g.ld, f.ld_dz = dg.ld, f.dtype = dt, f.w_layout = oi;
    return f;
}
static muon_gated_grad_input_args input_args(long rows, long in, long hid, int es, int dt, bool oi) {
    muon_gated_grad_input_args f{};
    const Buf dg = mat(rows, hid, es), du = mat(rows, hid, es), dx = mat(rows, in, es),
              wg = oi ? mat(hid, in, es) : mat(in, hid, es), wu = oi ? mat(hid, in, es) : mat(in, hid, es);
    f.dgate = dg.p, f.dup = du.p, f.w_gate = wg.p, f.w_up = wu.p, f.dx = dx.p, f.rows = rows, f.in = in, f.hidden = hid;
    f.ld_dz = dg.ld, f.ld_w = wg.ld, f.ld_dx = dx.ld, f.dtype = dt, f.w_layout = oi;
    return f;
}
static muon_gated_grad_weight_args weight_args(long rows, long in, long hid, int es, int dt, bool oi) {
    muon_gated_grad_weight_args f{};
    const Buf x = mat(rows, in, es), dg = mat(rows, hid, es), du = mat(rows, hid, es),
              wg = oi ? mat(hid, in, es) : mat(in, hid, es), wu = oi ? mat(hid, in, es) : mat(in, hid, es);
    f.x = x.p, f.dgate = dg.p, f.dup = du.p, f.dw_gate = wg.p, f.dw_up = wu.p, f.rows = rows, f.in = in, f.hidden = hid;
    f.ld_x = x.ld, f.ld_dz = dg.ld, f.ld_dw = wg.ld, f.dtype = f.dw_dtype = f.db_dtype = dt, f.w_layout = oi;
    return f;
}
static uint64_t g_step = 5;
static muon_dropout_mask mask(float p, bool step) { return muon_dropout_mask{p, 0, 0x123456789ABCull, 77, step ? &g_step : nullptr}; }

// A junction with everything it can have; kind 1 RMS, 2 layer norm.
static muon_blocknorm_args norm_args(long rows, long cols, int ss, int es, int st, int dt, int kind, bool branch) {
    muon_blocknorm_args f{};
    const Buf x = mat(rows, cols, ss), b = mat(rows, cols, es), s = mat(rows, cols, ss), y = mat(rows, cols, es);
    f.x = x.p, f.ld_x = x.ld, f.y = y.p, f.ld_y = y.ld, f.rows = rows, f.cols = cols, f.pre_norm = kind;
    f.residual_scale = 1.f, f.branch_scale = 0.5f, f.post_eps = f.pre_eps = 1e-5f;
    f.stream_dtype = st, f.dtype = dt, f.param_dtype = dt;
    f.pre_gain = vec(cols, es).p, f.pre_rstd = vec(rows, 4).f();
    if (kind == 2) f.pre_bias = vec(cols, es).p, f.pre_mean = vec(rows, 4).f();
    if (!branch) return f;
    f.branch = b.p, f.ld_branch = b.ld, f.s = s.p, f.ld_s = s.ld, f.post_norm = kind, f.residual_scale = 0.75f;
    f.post_gain = vec(cols, es).p, f.gate = vec(cols, es).p, f.post_rstd = vec(rows, 4).f();
    if (kind == 2) f.post_bias = vec(cols, es).p, f.post_mean = vec(rows, 4).f();
    f.drop = mask(0.25f, true);
    return f;
}
static muon_blocknorm_grad_args norm_grad_args(long rows, long cols, int ss, int es, int st, int dt, int kind, bool branch) {
    muon_blocknorm_grad_args f{};
    const Buf dy = mat(rows, cols, es), ds = mat(rows, cols, ss), s = mat(rows, cols, ss), b = mat(rows, cols, es),
              dx = mat(rows, cols, ss), db = mat(rows, cols, es);
    f.dy = dy.p, f.ld_dy = dy.ld, f.ds = ds.p, f.ld_ds = ds.ld, f.s = s.p, f.ld_s = s.ld, f.dx = dx.p, f.ld_dx = dx.ld;
    f.rows = rows, f.cols = cols, f.pre_norm = kind, f.residual_scale = 0.75f, f.branch_scale = 0.5f;
    f.stream_dtype = st, f.dtype = dt, f.param_dtype = dt;
    f.pre_gain = vec(cols, es).p, f.dpre_gain = vec(cols, es).p, f.pre_rstd = vec(rows, 4).f();
    if (kind == 2) f.dpre_bias = vec(cols, es).p, f.pre_mean = vec(rows, 4).f();
    if (!branch) return f;
    f.branch = b.p, f.ld_branch = b.ld, f.dbranch = db.p, f.ld_dbranch = db.ld, f.post_norm = kind;
    f.post_gain = vec(cols, es).p, f.dpost_gain = vec(cols, es).p, f.gate = vec(cols, es).p, f.dgate = vec(cols, es).p;
    f.post_rstd = vec(rows, 4).f();
    if (kind == 2) f.post_bias = vec(cols, es).p, f.dpost_bias = vec(cols, es).p, f.post_mean = vec(rows, 4).f();
    f.drop = mask(0.25f, true);
    return f;
}
static muon_dropout_args drop_args(long rows, long cols, int es, int dt) {
    muon_dropout_args f{};
    const Buf x = mat(rows, cols, es), y = mat(rows, cols, es), a = mat(rows, cols, es);
    f.x = x.p, f.y = y.p, f.add = a.p, f.ld_x = x.ld, f.ld_y = y.ld, f.ld_add = a.ld, f.rows = rows, f.cols = cols;
    f.dtype = dt, f.drop = mask(0.5f, false);
    return f;
}

// Calls that must be refused, with nothing enqueued: each case is a valid call
// with one thing changed.
static int refuse() {
    muon_handle* h = nullptr;
    if (muon_init(&h, 0, 0) != MUON_OK) return 3;
    long wrong = 0;
    const long before = emu_launches;
    auto expect = [&](const char* what, muon_status got, muon_status want) {
        if (got != want || emu_launches != before || (want != MUON_OK && !*muon_last_error(h))) {
            std::printf("%s: status %d, want %d, launches %ld, \"%s\"\n", what, int(got), int(want),
                        emu_launches - before, muon_last_error(h));
            ++wrong;
        }
    };
    const muon_status inv = MUON_ERR_INVALID_ARG, dty = MUON_ERR_DTYPE;
    auto off = [](const void* p) { return static_cast<const void*>(static_cast<const char*>(p) + 1); };
    // T(call, valid arguments): t(name, status, change)
    auto table = [&](auto call, auto ok) {
        expect("null arguments", call(h, nullptr, nullptr), inv);
        if (call(nullptr, &ok, nullptr) != inv) ++wrong;
        return [&, call, ok](const char* what, muon_status want, auto&& f) {
            auto a = ok;
            f(a);
            expect(what, call(h, &a, nullptr), want);
        };
    };
    const muon_act8 q = act8(4, 48), q2 = act8(4, 48);
    {
        muon_gated_args ok = gated_args(4, 40, 48, 2, MUON_BF16, false);
        auto t = table(muon_gated_forward, ok);
        const Buf z = mat(4, 48, 2), z2 = mat(4, 48, 2), b = vec(48, 2);
        t("dtype", dty, [](auto& a) { a.dtype = 2; });
        t("bias dtype", dty, [&](auto& a) { a.bias_up = b.p; a.bias_dtype = 9; });
        t("rows", inv, [](auto& a) { a.rows = -1; });
        t("many rows", inv, [](auto& a) { a.rows = int64_t(1) << 31; });
        t("in 0", inv, [](auto& a) { a.in = 0; });
        t("hidden", inv, [](auto& a) { a.hidden = (1 << 20) + 1; a.ld_w = a.ld_h = a.hidden; });
        t("tiles", inv, [](auto& a) { a.rows = (int64_t(1) << 31) - 1; a.hidden = 1 << 20; a.ld_w = a.ld_h = a.hidden; });
        t("activation", inv, [](auto& a) { a.activation = 4; });
        t("layout", inv, [](auto& a) { a.w_layout = 2; });
        t("reserved", inv, [](auto& a) { a.reserved = 1; });
        t("x", inv, [](auto& a) { a.x = nullptr; });
        t("w_up", inv, [](auto& a) { a.w_up = nullptr; });
        t("ld_w", inv, [](auto& a) { a.ld_w = 47; });
        t("ld_w of the other layout", inv, [](auto& a) { a.w_layout = 1; a.ld_w = 39; });
        t("misaligned", inv, [&](auto& a) { a.w_up = off(a.w_up); });
        t("h is x", inv, [](auto& a) { a.h = const_cast<void*>(a.x); });
        t("gate alone", inv, [&](auto& a) { a.gate = z.p; a.ld_z = 48; });
        t("gate is up", inv, [&](auto& a) { a.gate = a.up = z.p; a.ld_z = 48; });
        t("ld_z", inv, [&](auto& a) { a.gate = z.p; a.up = z2.p; a.ld_z = 47; });
        t("gate8 alone", inv, [&](auto& a) { a.gate8 = q; });
        t("gate8 is up8", inv, [&](auto& a) { a.gate8 = a.up8 = q; });
        t("gate and gate8", inv, [&](auto& a) { a.gate = z.p; a.up = z2.p; a.ld_z = 48; a.gate8 = q; a.up8 = q2; });
        t("exponents", inv, [&](auto& a) { a.gate8 = q; a.up8 = q2; a.up8.exponents = nullptr; });
        t("no rows", MUON_OK, [](auto& a) { a.rows = 0; a.x = nullptr; a.h = nullptr; });
    }
    {
        muon_gated_grad_hidden_args ok = hidden_args(4, 48, 40, 2, MUON_BF16, false);
        auto t = table(muon_gated_grad_hidden, ok);
        t("dtype", dty, [](auto& a) { a.dtype = -1; });
        t("activation", inv, [](auto& a) { a.activation = -1; });
        t("layout", inv, [](auto& a) { a.w_layout = -1; });
        t("reserved", inv, [](auto& a) { a.reserved = 3; });
        t("no pre-activation", inv, [](auto& a) { a.gate = a.up = nullptr; });
        t("up alone", inv, [](auto& a) { a.gate = nullptr; });
        t("both forms", inv, [&](auto& a) { a.gate8 = q; a.up8 = q2; });
        t("dup", inv, [](auto& a) { a.dup = nullptr; });
        t("dup is dgate", inv, [](auto& a) { a.dup = a.dgate; });
        t("dgate is gate", inv, [](auto& a) { a.dgate = const_cast<void*>(a.gate); });
        t("w_down", inv, [](auto& a) { a.w_down = nullptr; });
        t("ld_dz", inv, [](auto& a) { a.ld_dz = 40; });
        t("out", inv, [](auto& a) { a.out = 0; });
        t("no rows", MUON_OK, [](auto& a) { a.rows = 0; a.dy = nullptr; a.dgate = a.dup = nullptr; a.gate = a.up = nullptr; });
    }
    {
        muon_gated_grad_input_args ok = input_args(4, 40, 48, 2, MUON_BF16, true);
        auto t = table(muon_gated_grad_input, ok);
        t("dtype", dty, [](auto& a) { a.dtype = 5; });
        t("reserved", inv, [](auto& a) { a.reserved = 3; });
        t("dup", inv, [](auto& a) { a.dup = nullptr; });
        t("dx is dup", inv, [](auto& a) { a.dx = const_cast<void*>(a.dup); });
        t("dx is add of another ld", inv, [](auto& a) { a.add = a.dx; a.ld_add = a.ld_dx + 8; });
        t("w_gate", inv, [](auto& a) { a.w_gate = nullptr; });
        t("ld_w", inv, [](auto& a) { a.ld_w = 39; });
        t("misaligned dup", inv, [&](auto& a) { a.dup = off(a.dup); });
        t("no rows", MUON_OK, [](auto& a) { a.rows = 0; a.dgate = a.dup = nullptr; a.dx = nullptr; });
    }
    {
        muon_gated_grad_weight_args ok = weight_args(4, 48, 40, 2, MUON_BF16, false);
        auto t = table(muon_gated_grad_weight, ok);
        t("dtype", dty, [](auto& a) { a.dtype = 5; });
        t("dw dtype", dty, [](auto& a) { a.dw_dtype = 5; });
        t("db dtype", dty, [](auto& a) { a.db_up = a.dw_gate; a.db_dtype = 5; });
        t("accumulate", inv, [](auto& a) { a.accumulate = 2; });
        t("x and x8", inv, [&](auto& a) { a.x8 = q; });
        t("no x", inv, [](auto& a) { a.x = nullptr; });
        t("dw_up", inv, [](auto& a) { a.dw_up = nullptr; });
        t("dw_up is dw_gate", inv, [](auto& a) { a.dw_up = a.dw_gate; });
        t("dw is dup", inv, [](auto& a) { a.dw_up = const_cast<void*>(a.dup); });
        t("db is dw", inv, [](auto& a) { a.db_up = a.dw_gate; });
        t("ld_dw", inv, [](auto& a) { a.ld_dw = 39; });
    }
    {
        muon_dropout_args ok = drop_args(4, 40, 2, MUON_BF16);
        auto t = table(muon_dropout, ok);
        t("dtype", dty, [](auto& a) { a.dtype = 5; });
        t("p under 0", inv, [](auto& a) { a.drop.p = -0.01f; });
        t("p over 1", inv, [](auto& a) { a.drop.p = 1.01f; });
        t("p nan", inv, [](auto& a) { a.drop.p = std::nanf(""); });
        t("mask reserved", inv, [](auto& a) { a.drop.reserved = 1; });
        t("reserved", inv, [](auto& a) { a.reserved = 1; });
        t("step", inv, [](auto& a) { a.drop.step = reinterpret_cast<const uint64_t*>(reinterpret_cast<const char*>(&g_step) + 4); });
        t("y", inv, [](auto& a) { a.y = nullptr; });
        t("y is x of another ld", inv, [](auto& a) { a.y = const_cast<void*>(a.x); a.ld_y = 48; });
        t("y is add of another ld", inv, [](auto& a) { a.y = const_cast<void*>(a.add); a.ld_y = 48; });
        t("cols", inv, [](auto& a) { a.cols = 0; });
        t("no rows", MUON_OK, [](auto& a) { a.rows = 0; a.x = nullptr; a.y = nullptr; });
    }
    {
        muon_blocknorm_args ok = norm_args(4, 40, 2, 2, MUON_BF16, MUON_BF16, 2, true);
        auto t = table(muon_blocknorm_forward, ok);
        t("dtype", dty, [](auto& a) { a.dtype = 5; });
        t("stream dtype", dty, [](auto& a) { a.stream_dtype = 5; });
        t("param dtype", dty, [](auto& a) { a.param_dtype = 5; });
        t("bf16 stream, float32 blocks", dty, [](auto& a) { a.dtype = MUON_F32; });
        t("post norm", inv, [](auto& a) { a.post_norm = 3; });
        t("pre norm", inv, [](auto& a) { a.pre_norm = -1; });
        t("scale", inv, [](auto& a) { a.branch_scale = INFINITY; });
        t("residual scale", inv, [](auto& a) { a.residual_scale = std::nanf(""); });
        t("eps", inv, [](auto& a) { a.post_eps = -1.f; });
        t("p", inv, [](auto& a) { a.drop.p = 2.f; });
        t("x", inv, [](auto& a) { a.x = nullptr; });
        t("s", inv, [](auto& a) { a.s = nullptr; });
        t("y", inv, [](auto& a) { a.y = nullptr; });
        t("y without pre norm", inv, [](auto& a) { a.pre_norm = 0; a.pre_gain = a.pre_bias = nullptr; a.pre_mean = a.pre_rstd = nullptr; });
        t("gain without pre norm", inv, [](auto& a) { a.pre_norm = 0; a.pre_bias = nullptr; a.y = nullptr; a.pre_mean = a.pre_rstd = nullptr; });
        t("gain without post norm", inv, [](auto& a) { a.post_norm = 0; a.post_bias = nullptr; a.post_mean = a.post_rstd = nullptr; });
        t("bias of an RMS norm", inv, [](auto& a) { a.post_norm = 1; a.post_mean = nullptr; });
        t("pre bias of an RMS norm", inv, [](auto& a) { a.pre_norm = 1; a.pre_mean = nullptr; });
        t("mean of an RMS norm", inv, [](auto& a) { a.pre_norm = 1; a.pre_bias = nullptr; });
        t("no branch", inv, [](auto& a) { a.branch = nullptr; });
        t("s is x of another ld", inv, [](auto& a) { a.s = const_cast<void*>(a.x); a.ld_s = 48; });
        t("s is branch", inv, [](auto& a) { a.s = const_cast<void*>(a.branch); });
        t("y is s", inv, [](auto& a) { a.y = a.s; });
        t("y is x", inv, [](auto& a) { a.y = const_cast<void*>(a.x); });
        t("misaligned branch", inv, [&](auto& a) { a.branch = off(a.branch); });
        t("misaligned gate", inv, [&](auto& a) { a.gate = off(a.gate); });
        t("ld_branch", inv, [](auto& a) { a.ld_branch = 39; });
        t("y8", inv, [&](auto& a) { a.y8 = q; a.y8.exponents = nullptr; });
        t("cols", inv, [](auto& a) { a.cols = (1 << 20) + 1; a.ld_x = a.ld_branch = a.ld_s = a.ld_y = a.cols; });
        t("reserved", inv, [](auto& a) { a.reserved = 1; });
        t("no rows", MUON_OK, [](auto& a) { a.rows = 0; a.x = a.branch = nullptr; a.s = a.y = nullptr; });
    }
    {
        muon_blocknorm_grad_args ok = norm_grad_args(4, 40, 2, 2, MUON_BF16, MUON_BF16, 2, true);
        auto t = table(muon_blocknorm_backward, ok);
        t("dtype", dty, [](auto& a) { a.dtype = 5; });
        t("bf16 stream, float32 blocks", dty, [](auto& a) { a.dtype = MUON_F32; });
        t("accumulate", inv, [](auto& a) { a.accumulate = -1; });
        t("dx", inv, [](auto& a) { a.dx = nullptr; });
        t("dy", inv, [](auto& a) { a.dy = nullptr; });
        t("s", inv, [](auto& a) { a.s = nullptr; });
        t("pre_rstd", inv, [](auto& a) { a.pre_rstd = nullptr; });
        t("pre_mean", inv, [](auto& a) { a.pre_mean = nullptr; });
        t("post_mean", inv, [](auto& a) { a.post_mean = nullptr; });
        t("branch", inv, [](auto& a) { a.branch = nullptr; });
        t("dbranch", inv, [](auto& a) { a.dbranch = nullptr; });
        t("dgate without gate", inv, [](auto& a) { a.gate = nullptr; });
        t("dpost_gain without gain", inv, [](auto& a) { a.post_gain = nullptr; });
        t("dpost_bias without bias", inv, [](auto& a) { a.post_bias = nullptr; });
        t("dpre_gain without gain", inv, [](auto& a) { a.pre_gain = nullptr; });
        t("dpre_bias of an RMS norm", inv, [](auto& a) { a.pre_norm = 1; });
        t("nothing behind", inv, [](auto& a) { a.pre_norm = 0; a.dy = nullptr; a.pre_gain = nullptr; a.dpre_gain = a.dpre_bias = nullptr; a.ds = nullptr; });
        t("dx is ds of another ld", inv, [](auto& a) { a.dx = const_cast<void*>(a.ds); a.ld_dx = 48; });
        t("dx is s", inv, [](auto& a) { a.dx = const_cast<void*>(a.s); });
        t("dbranch is branch", inv, [](auto& a) { a.dbranch = const_cast<void*>(a.branch); });
        t("dgate is gate", inv, [](auto& a) { a.dgate = const_cast<void*>(a.gate); });
        t("ld_ds", inv, [](auto& a) { a.ld_ds = 39; });
        t("reserved", inv, [](auto& a) { a.reserved = 1; });
    }
    muon_destroy(h);
    // an allocation that fails: the call is refused and enqueues nothing
    if (muon_init(&h, 0, MUON_INIT_FAIL_ALLOC) != MUON_OK) return 3;
    muon_blocknorm_grad_args a = norm_grad_args(4, 40, 2, 2, MUON_BF16, MUON_BF16, 1, true);
    expect("out of memory", muon_blocknorm_backward(h, &a, nullptr), MUON_ERR_OOM);
    muon_gated_args g = gated_args(4, 41, 48, 2, MUON_BF16, false);   // a ragged operand to re-lay
    expect("out of memory", muon_gated_forward(h, &g, nullptr), MUON_ERR_OOM);
    muon_destroy(h);
    for (const Buf& t : bufs) std::free(t.alloc);
    std::printf("refusals wrong %ld\n", wrong);
    return wrong ? 6 : 0;
}

int main(int argc, char** argv) {
    if (argc == 2 && std::string(argv[1]) == "refuse") return refuse();
    if (argc < 9) return 2;
    emu_verbose = std::getenv("EMU_VERBOSE") != nullptr;
    const std::string op = argv[1];
    const long rows = std::atol(argv[2]), A = std::atol(argv[3]), B = std::atol(argv[4]);
    const int types = std::atoi(argv[5]), flags = std::atoi(argv[6]);
    const int dt = types == 1 ? MUON_F32 : MUON_BF16, st = types == 0 ? MUON_BF16 : MUON_F32;
    const int es = dt == MUON_BF16 ? 2 : 4, ss = st == MUON_BF16 ? 2 : 4;
    g_pad = std::atol(argv[7]);
    g_shift = std::atol(argv[8]);
    const bool oi = flags & 1, q8 = flags & 2, bare = flags & 4, branch = !(flags & 16), place = flags & 32;
    const int kind = flags & 8 ? 2 : 1;
    muon_handle* h = nullptr;
    if (muon_init(&h, 0, 0) != MUON_OK) return 3;
    int rc = 0;
    auto run = [&](const char* what, muon_status s) {
        std::printf("%s %d (%s)\n", what, int(s), muon_last_error(h));
        if (s != MUON_OK) rc = 4;
    };
    if (op == "gated") {
        muon_gated_args f = gated_args(rows, A, B, es, dt, oi);
        const Buf z = mat(rows, B, es), z2 = mat(rows, B, es);
        if (!bare) f.bias_gate = vec(B, es).p, f.bias_up = vec(B, es).p;
        if (q8) f.gate8 = act8(rows, B), f.up8 = act8(rows, B);
        else if (!bare) f.gate = z.p, f.up = z2.p, f.ld_z = z.ld;
        run("forward", muon_gated_forward(h, &f, nullptr));
        muon_gated_grad_hidden_args d = hidden_args(rows, B, A, es, dt, oi);
        const Buf ho = mat(rows, B, es);
        d.activation = MUON_GATE_RELU;
        if (!bare) d.h = ho.p, d.ld_h = ho.ld, d.activation = MUON_GATE_GELU;
        if (q8) d.gate = d.up = nullptr, d.gate8 = act8(rows, B), d.up8 = act8(rows, B);
        run("grad hidden", muon_gated_grad_hidden(h, &d, nullptr));
        muon_gated_grad_input_args i = input_args(rows, A, B, es, dt, oi);
        const Buf add = mat(rows, A, es);
        if (place) i.add = i.dx, i.ld_add = i.ld_dx;
        else if (!bare) i.add = add.p, i.ld_add = add.ld;
        run("grad input", muon_gated_grad_input(h, &i, nullptr));
        muon_gated_grad_weight_args w = weight_args(rows, A, B, es, dt, oi);
        if (q8) w.x = nullptr, w.x8 = act8(rows, A);
        if (!bare) w.db_gate = vec(B, es).p, w.db_up = vec(B, es).p, w.accumulate = 1;
        run("grad weight", muon_gated_grad_weight(h, &w, nullptr));
        w.db_gate = nullptr, w.db_up = vec(B, 4).p, w.db_dtype = MUON_F32, w.accumulate = 0;
        run("grad weight, one bias", muon_gated_grad_weight(h, &w, nullptr));
    } else if (op == "norm") {
        muon_blocknorm_args f = norm_args(rows, A, ss, es, st, dt, kind, branch);
        if (q8) f.y8 = act8(rows, A);
        if (bare) f.gate = f.post_gain = f.post_bias = f.pre_gain = f.pre_bias = nullptr, f.drop = muon_dropout_mask{};
        if (bare) f.post_rstd = f.post_mean = f.pre_rstd = f.pre_mean = nullptr;
        if (place && branch) f.s = const_cast<void*>(f.x), f.ld_s = f.ld_x;
        run("forward", muon_blocknorm_forward(h, &f, nullptr));
        muon_blocknorm_grad_args d = norm_grad_args(rows, A, ss, es, st, dt, kind, branch);
        d.accumulate = !bare;
        if (bare) {
            d.gate = d.post_gain = d.post_bias = d.pre_gain = nullptr;
            d.dgate = d.dpost_gain = d.dpost_bias = d.dpre_gain = nullptr;
            d.ds = nullptr, d.drop = muon_dropout_mask{};
        }
        if (place && d.ds) d.dx = const_cast<void*>(d.ds), d.ld_dx = d.ld_ds;
        run("backward", muon_blocknorm_backward(h, &d, nullptr));
        if (branch) {   // the end of the stack: no norm behind the junction
            f.pre_norm = 0, f.y = nullptr, f.pre_gain = f.pre_bias = nullptr, f.pre_mean = f.pre_rstd = nullptr;
            f.y8 = muon_act8{};
            run("forward, no norm behind", muon_blocknorm_forward(h, &f, nullptr));
            if (d.ds) {
                d.pre_norm = 0, d.dy = d.s = nullptr, d.pre_gain = nullptr, d.dpre_gain = d.dpre_bias = nullptr;
                run("backward, no norm behind", muon_blocknorm_backward(h, &d, nullptr));
            }
        }
    } else {
        muon_dropout_args f = drop_args(rows, A, es, dt);
        if (bare) f.add = nullptr;
        if (place) f.y = const_cast<void*>(f.x), f.ld_y = f.ld_x;
        run("dropout", muon_dropout(h, &f, nullptr));
    }
    const long bad = damaged();
    std::printf("damaged padding bytes %ld\n", bad);
    muon_destroy(h);
    for (const Buf& b : bufs) std::free(b.alloc);
    return bad ? 5 : rc;
}
