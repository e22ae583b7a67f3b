// Test infrastructure: runs the layer operators of the library, built against
// the CPU stand-in of HIP, on exactly sized host buffers, so AddressSanitizer
// reports any access outside them.  Usage:
//   emu_layers_driver OP ROWS A B DTYPE FLAGS PAD SHIFT | emu_layers_driver refuse
// OP ln | lin | act; A, B = cols, - or in, out; DTYPE 0 bf16, 1 f32; FLAGS bit 0
// weight layout out x in, bit 1 8-bit checkpoints, bit 2 without the optional
// arguments; PAD extra elements per row, SHIFT elements by which every buffer
// starts past its allocation.  The bytes between rows are checked to keep their
// value.
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
};
static std::vector<Buf> bufs;
static long g_pad, g_shift;

static Buf mat(long rows, long cols, int es) {
    Buf b;
    b.rows = rows;
    b.cols = cols;
    b.ld = cols + g_pad;
    b.es = es;
    const long n = rows > 0 ? (rows - 1) * b.ld + cols + g_shift : g_shift;
    b.alloc = static_cast<char*>(std::malloc(n * es > 0 ? n * es : 1));
    b.p = b.alloc + g_shift * es;
    for (long r = 0; r < rows; ++r)
        for (long c = 0; c < (r + 1 < rows ? b.ld : cols); ++c) {
            char* q = b.p + (r * b.ld + c) * es;
            if (c >= cols) {
                std::memset(q, 0x5A, es);
            } else if (es == 4) {
                const float f = float((r * 7 + c * 3) % 13 - 6) * 0.25f;
                std::memcpy(q, &f, 4);
            } else if (es == 2) {
                const float f = float((r * 7 + c * 3) % 13 - 6) * 0.25f;
                uint32_t u;
                std::memcpy(&u, &f, 4);
                const uint16_t h = uint16_t(u >> 16);
                std::memcpy(q, &h, 2);
            } else {
                *q = char(120 + (r + c) % 8);   // as a code or as an exponent byte
            }
        }
    bufs.push_back(b);
    return b;
}
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

// Calls that must be refused, with nothing enqueued: each case is a valid call
// with one thing changed.
static int refuse() {
    muon_handle* h = nullptr;
    if (muon_init(&h, 0, 0) != MUON_OK) return 3;
    const Buf x = mat(4, 40, 2), y = mat(4, 48, 2), w = mat(40, 48, 2), g = mat(1, 48, 2), b = mat(1, 48, 2),
              r = mat(4, 48, 2), s0 = mat(1, 4, 4), s1 = mat(1, 4, 4), o = mat(4, 40, 2), dw = mat(40, 48, 2);
    const muon_act8 q40 = act8(4, 40), q48 = act8(4, 48);
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
    {
        muon_layernorm_args ok{};
        ok.x = x.p, ok.gain = g.p, ok.y = o.p, ok.rows = 4, ok.cols = 40, ok.ld_x = x.ld, ok.ld_y = o.ld;
        auto t = [&](const char* what, muon_status want, auto&& f) {
            muon_layernorm_args a = ok;
            f(a);
            expect(what, muon_layernorm_forward(h, &a, nullptr), want);
        };
        expect("ln null", muon_layernorm_forward(h, nullptr, nullptr), inv);
        if (muon_layernorm_forward(nullptr, &ok, nullptr) != inv) ++wrong;
        t("ln dtype", dty, [](auto& a) { a.dtype = 7; });
        t("ln param dtype", dty, [](auto& a) { a.param_dtype = -1; });
        t("ln rows", inv, [](auto& a) { a.rows = -1; });
        t("ln many rows", inv, [](auto& a) { a.rows = int64_t(1) << 31; });
        t("ln cols 0", inv, [](auto& a) { a.cols = 0; });
        t("ln cols", inv, [](auto& a) { a.cols = (1 << 20) + 1; a.ld_x = a.ld_y = a.cols; });
        t("ln ld", inv, [](auto& a) { a.ld_x = 39; });
        t("ln x", inv, [](auto& a) { a.x = nullptr; });
        t("ln gain", inv, [](auto& a) { a.gain = nullptr; });
        t("ln in place", inv, [](auto& a) { a.y = const_cast<void*>(a.x); });
        t("ln eps", inv, [](auto& a) { a.eps = -1.f; });
        t("ln eps nan", inv, [](auto& a) { a.eps = std::nanf(""); });
        t("ln reserved", inv, [](auto& a) { a.reserved = 1; });
        t("ln mean is rstd", inv, [&](auto& a) { a.mean = a.rstd = reinterpret_cast<float*>(s0.p); });
        t("ln misaligned x", inv, [](auto& a) { a.x = static_cast<const char*>(a.x) + 1; });
        t("ln y8 without exponents", inv, [&](auto& a) { a.y8 = q40; a.y8.exponents = nullptr; });
        t("ln y8 without codes", inv, [&](auto& a) { a.y8 = q40; a.y8.codes = nullptr; });
        t("ln y8 ld", inv, [&](auto& a) { a.y8 = q40; a.y8.ld_codes = 39; });
        t("ln y8 ld exponents", inv, [&](auto& a) { a.y8 = q40; a.y8.ld_exponents = 1; });
        t("ln no rows", MUON_OK, [](auto& a) { a.rows = 0; a.x = nullptr; a.y = nullptr; });
    }
    {
        muon_layernorm_grad_args ok{};
        ok.dy = r.p, ok.x = x.p, ok.gain = g.p, ok.mean = reinterpret_cast<float*>(s0.p);
        ok.rstd = reinterpret_cast<float*>(s1.p), ok.dx = o.p, ok.dgain = b.p, ok.rows = 4, ok.cols = 40;
        ok.ld_dy = r.ld, ok.ld_x = x.ld, ok.ld_dx = o.ld;
        auto t = [&](const char* what, muon_status want, auto&& f) {
            muon_layernorm_grad_args a = ok;
            f(a);
            expect(what, muon_layernorm_backward(h, &a, nullptr), want);
        };
        expect("ln grad null", muon_layernorm_backward(h, nullptr, nullptr), inv);
        t("ln grad dtype", dty, [](auto& a) { a.dtype = 2; });
        t("ln grad accumulate", inv, [](auto& a) { a.accumulate = 2; });
        t("ln grad reserved", inv, [](auto& a) { a.reserved = 1; });
        t("ln grad mean", inv, [](auto& a) { a.mean = nullptr; });
        t("ln grad dgain", inv, [](auto& a) { a.dgain = nullptr; });
        t("ln grad dx is dy", inv, [](auto& a) { a.dx = const_cast<void*>(a.dy); });
        t("ln grad dgain is gain", inv, [](auto& a) { a.dgain = const_cast<void*>(a.gain); });
        t("ln grad dbias is dgain", inv, [](auto& a) { a.dbias = a.dgain; });
        t("ln grad add is dx, other ld", inv, [](auto& a) { a.add = a.dx; a.ld_add = a.ld_dx + 8; });
        t("ln grad add ld", inv, [&](auto& a) { a.add = y.p; a.ld_add = 3; });
    }
    {
        muon_linear_args ok{};
        ok.x = x.p, ok.w = w.p, ok.y = y.p, ok.rows = 4, ok.in = 40, ok.out = 48, ok.ld_x = x.ld, ok.ld_w = w.ld;
        ok.ld_y = y.ld;
        auto t = [&](const char* what, muon_status want, auto&& f) {
            muon_linear_args a = ok;
            f(a);
            expect(what, muon_linear_forward(h, &a, nullptr), want);
        };
        expect("lin null", muon_linear_forward(h, nullptr, nullptr), inv);
        t("lin dtype", dty, [](auto& a) { a.dtype = 2; });
        t("lin bias dtype", dty, [&](auto& a) { a.bias = b.p; a.bias_dtype = 2; });
        t("lin act", inv, [](auto& a) { a.activation = 3; });
        t("lin layout", inv, [](auto& a) { a.w_layout = 2; });
        t("lin out x in ld", inv, [](auto& a) { a.w_layout = 1; a.ld_w = 39; });
        t("lin ld w", inv, [](auto& a) { a.ld_w = 47; });
        t("lin in 0", inv, [](auto& a) { a.in = 0; });
        t("lin out", inv, [](auto& a) { a.out = (1 << 20) + 1; });
        t("lin huge", inv, [](auto& a) { a.rows = (int64_t(1) << 31) - 1; a.out = 1 << 20; a.ld_w = a.ld_y = a.out; });
        t("lin y is x", inv, [](auto& a) { a.y = const_cast<void*>(a.x); a.out = 40; a.ld_y = a.ld_x; });
        t("lin y is w", inv, [](auto& a) { a.y = const_cast<void*>(a.w); });
        t("lin residual is y, other ld", inv, [](auto& a) { a.residual = a.y; a.ld_residual = a.ld_y + 8; });
        t("lin z and z8", inv, [&](auto& a) { a.z = r.p; a.ld_z = r.ld; a.z8 = q48; });
        t("lin z is y", inv, [](auto& a) { a.z = a.y; a.ld_z = a.ld_y; });
        t("lin w", inv, [](auto& a) { a.w = nullptr; });
        t("lin reserved", inv, [](auto& a) { a.reserved = 5; });
        t("lin no rows", MUON_OK, [](auto& a) { a.rows = 0; a.x = nullptr; a.y = nullptr; });
    }
    {
        muon_linear_grad_input_args ok{};
        ok.dy = r.p, ok.w = w.p, ok.dx = o.p, ok.rows = 4, ok.in = 40, ok.out = 48, ok.ld_dy = r.ld, ok.ld_w = w.ld;
        ok.ld_dx = o.ld;
        auto t = [&](const char* what, muon_status want, auto&& f) {
            muon_linear_grad_input_args a = ok;
            f(a);
            expect(what, muon_linear_grad_input(h, &a, nullptr), want);
        };
        expect("dx null", muon_linear_grad_input(h, nullptr, nullptr), inv);
        t("dx dtype", dty, [](auto& a) { a.dtype = 9; });
        t("dx activation without z", inv, [](auto& a) { a.activation = 1; });
        t("dx act_out without z", inv, [&](auto& a) { a.act_out = x.p; a.ld_act_out = x.ld; });
        t("dx z and z8", inv, [&](auto& a) { a.z = x.p; a.ld_z = x.ld; a.z8 = q40; });
        t("dx is z", inv, [](auto& a) { a.z = a.dx; a.ld_z = a.ld_dx; });
        t("dx z8 ld", inv, [&](auto& a) { a.z8 = q40; a.z8.ld_codes = 8; });
        t("dx add is dx, other ld", inv, [](auto& a) { a.add = a.dx; a.ld_add = a.ld_dx + 1; });
        t("dx dy", inv, [](auto& a) { a.dy = nullptr; });
    }
    {
        muon_linear_grad_weight_args ok{};
        ok.x = x.p, ok.dy = r.p, ok.dw = dw.p, ok.rows = 4, ok.in = 40, ok.out = 48, ok.ld_x = x.ld, ok.ld_dy = r.ld;
        ok.ld_dw = dw.ld;
        auto t = [&](const char* what, muon_status want, auto&& f) {
            muon_linear_grad_weight_args a = ok;
            f(a);
            expect(what, muon_linear_grad_weight(h, &a, nullptr), want);
        };
        expect("dw null", muon_linear_grad_weight(h, nullptr, nullptr), inv);
        t("dw dtype", dty, [](auto& a) { a.dw_dtype = 2; });
        t("db dtype", dty, [&](auto& a) { a.db = b.p; a.db_dtype = 2; });
        t("dw x and x8", inv, [&](auto& a) { a.x8 = q40; });
        t("dw without x", inv, [](auto& a) { a.x = nullptr; });
        t("dw accumulate", inv, [](auto& a) { a.accumulate = -1; });
        t("dw out x in ld", inv, [](auto& a) { a.w_layout = 1; a.ld_dw = 39; });
        t("dw is dy", inv, [](auto& a) { a.dw = const_cast<void*>(a.dy); });
        t("dw is db", inv, [](auto& a) { a.db = a.dw; });
    }
    {
        expect("encode null", muon_act_encode(h, x.p, 4, 40, 40, MUON_BF16, nullptr, nullptr), inv);
        expect("encode dtype", muon_act_encode(h, x.p, 4, 40, 40, 5, &q40, nullptr), dty);
        expect("encode x", muon_act_encode(h, nullptr, 4, 40, 40, MUON_BF16, &q40, nullptr), inv);
        expect("encode ld", muon_act_encode(h, x.p, 4, 40, 39, MUON_BF16, &q40, nullptr), inv);
        expect("encode codes ld", muon_act_encode(h, x.p, 4, 48, 48, MUON_BF16, &q40, nullptr), inv);
        expect("encode in place", muon_act_encode(h, q40.codes, 4, 40, 40, MUON_BF16, &q40, nullptr), inv);
        expect("encode no rows", muon_act_encode(h, nullptr, 0, 40, 40, MUON_BF16, &q40, nullptr), MUON_OK);
        expect("decode y", muon_act_decode(h, &q40, nullptr, 4, 40, 40, MUON_BF16, nullptr), inv);
        expect("decode in place", muon_act_decode(h, &q40, q40.codes, 4, 40, 40, MUON_BF16, nullptr), inv);
        expect("decode rows", muon_act_decode(h, &q40, o.p, -4, 40, 40, MUON_BF16, nullptr), inv);
    }
    muon_destroy(h);
    // an allocation that fails: the call is refused and enqueues nothing
    if (muon_init(&h, 0, MUON_INIT_FAIL_ALLOC) != MUON_OK) return 3;
    muon_layernorm_grad_args a{};
    a.dy = r.p, a.x = x.p, a.gain = g.p, a.mean = reinterpret_cast<float*>(s0.p), a.rstd = reinterpret_cast<float*>(s1.p);
    a.dx = o.p, a.dgain = b.p, a.rows = 4, a.cols = 40, a.ld_dy = r.ld, a.ld_x = x.ld, a.ld_dx = o.ld;
    expect("out of memory", muon_layernorm_backward(h, &a, nullptr), MUON_ERR_OOM);
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
    const int dt = std::atoi(argv[5]), flags = std::atoi(argv[6]), es = dt == MUON_BF16 ? 2 : 4;
    g_pad = std::atol(argv[7]);
    g_shift = std::atol(argv[8]);
    const bool oi = flags & 1, q8 = flags & 2, bare = flags & 4;
    muon_handle* h = nullptr;
    if (muon_init(&h, 0, 0) != MUON_OK) return 3;
    int st = 0;
    auto run = [&](const char* what, muon_status s) {
        std::printf("%s %d (%s)\n", what, int(s), muon_last_error(h));
        if (s != MUON_OK) st = 4;
    };
    if (op == "ln") {
        const Buf x = mat(rows, A, es), y = mat(rows, A, es), g = mat(1, A, es), b = mat(1, A, es),
                  mean = mat(1, rows, 4), rstd = mat(1, rows, 4);
        muon_layernorm_args f{};
        f.x = x.p, f.gain = g.p, f.y = y.p, f.rows = rows, f.cols = A, f.ld_x = x.ld, f.ld_y = y.ld;
        f.mean = reinterpret_cast<float*>(mean.p), f.rstd = reinterpret_cast<float*>(rstd.p);
        f.dtype = f.param_dtype = dt, f.eps = 1e-5f;
        if (!bare) f.bias = b.p;
        if (q8) f.y8 = act8(rows, A);
        run("forward", muon_layernorm_forward(h, &f, nullptr));
        const Buf dy = mat(rows, A, es), dx = mat(rows, A, es), dg = mat(1, A, es), db = mat(1, A, es),
                  add = mat(rows, A, es);
        muon_layernorm_grad_args d{};
        d.dy = dy.p, d.x = x.p, d.gain = g.p, d.mean = f.mean, d.rstd = f.rstd, d.dx = dx.p, d.dgain = dg.p;
        d.rows = rows, d.cols = A, d.ld_dy = dy.ld, d.ld_x = x.ld, d.ld_dx = dx.ld, d.dtype = d.param_dtype = dt;
        if (!bare) d.dbias = db.p, d.add = add.p, d.ld_add = add.ld, d.accumulate = 1;
        run("backward", muon_layernorm_backward(h, &d, nullptr));
    } else if (op == "lin") {
        const Buf x = mat(rows, A, es), y = mat(rows, B, es), w = oi ? mat(B, A, es) : mat(A, B, es), b = mat(1, B, es),
                  res = mat(rows, B, es), z = mat(rows, B, es), zi = mat(rows, A, es);
        muon_linear_args f{};
        f.x = x.p, f.w = w.p, f.y = y.p, f.rows = rows, f.in = A, f.out = B, f.ld_x = x.ld, f.ld_w = w.ld, f.ld_y = y.ld;
        f.dtype = f.bias_dtype = dt, f.w_layout = oi, f.activation = MUON_ACT_GELU;
        if (!bare) f.bias = b.p, f.residual = res.p, f.ld_residual = res.ld;
        if (q8) f.z8 = act8(rows, B);
        else if (!bare) f.z = z.p, f.ld_z = z.ld;
        run("forward", muon_linear_forward(h, &f, nullptr));
        const Buf dy = mat(rows, B, es), dx = mat(rows, A, es), add = mat(rows, A, es), ao = mat(rows, A, es);
        muon_linear_grad_input_args d{};
        d.dy = dy.p, d.w = w.p, d.dx = dx.p, d.rows = rows, d.in = A, d.out = B;
        d.ld_dy = dy.ld, d.ld_w = w.ld, d.ld_dx = dx.ld, d.dtype = dt, d.w_layout = oi;
        if (q8) d.z8 = act8(rows, A);
        else if (!bare) d.z = zi.p, d.ld_z = zi.ld;
        if (q8 || !bare) d.activation = MUON_ACT_RELU_SQ, d.act_out = ao.p, d.ld_act_out = ao.ld;
        if (!bare) d.add = add.p, d.ld_add = add.ld;
        run("grad input", muon_linear_grad_input(h, &d, nullptr));
        const Buf dw = oi ? mat(B, A, es) : mat(A, B, es), db = mat(1, B, es);
        muon_linear_grad_weight_args v{};
        v.dy = dy.p, v.dw = dw.p, v.rows = rows, v.in = A, v.out = B, v.ld_dy = dy.ld, v.ld_dw = dw.ld;
        v.dtype = v.dw_dtype = v.db_dtype = dt, v.w_layout = oi;
        if (q8) v.x8 = act8(rows, A);
        else v.x = x.p, v.ld_x = x.ld;
        if (!bare) v.db = db.p, v.accumulate = 1;
        run("grad weight", muon_linear_grad_weight(h, &v, nullptr));
    } else {
        const Buf x = mat(rows, A, es), y = mat(rows, A, es);
        const muon_act8 q = act8(rows, A);
        run("encode", muon_act_encode(h, x.p, rows, A, x.ld, dt, &q, nullptr));
        run("decode", muon_act_decode(h, &q, y.p, rows, A, y.ld, dt, nullptr));
    }
    const long bad = damaged();
    std::printf("damaged padding bytes %ld\n", bad);
    muon_destroy(h);
    for (const Buf& b : bufs) std::free(b.alloc);
    return bad ? 5 : st;
}
