// Test infrastructure: makes layer calls against the launch-recording stand-in
// of HIP.  One command a line on standard input, one JSON object a line out:
//   new                      a fresh handle
//   limit BYTES              larger allocations fail (0: none does)
//   OP ROWS A B [WORD ...]   a call: ln lngrad (A columns) | fwd dx dw (A in, B out) | enc dec
// WORDs: f32; oi (weight out x in); bias res z z8 act=N actout add acc db x8 y8
// (optional arguments); dw=N (dtype of dw); shift=N (every matrix starts N
// elements past a 16-byte boundary); pad=N (elements between rows); null (every
// per-row pointer is null, as an empty tensor's is); capture (on a capturing
// stream).  Addresses are made up and never read.
#include <hip/hip_runtime.h>

#include <iostream>
#include <sstream>
#include <string>

#include "muon.h"

emu_idx threadIdx, blockIdx;
dim3 gridDim, blockDim;
long emu_launches = 0;
int emu_verbose = 0;

int main() {
    muon_handle* h = nullptr;
    if (muon_init(&h, 0, 0) != MUON_OK) return 3;
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string op, word;
        in >> op;
        if (op == "new") {
            muon_destroy(h);
            if (muon_init(&h, 0, 0) != MUON_OK) return 3;
            continue;
        }
        if (op == "limit") {
            size_t n = 0;
            in >> n;
            emu_limit = n ? n : ~size_t(0);
            continue;
        }
        int64_t rows = 0, A = 0, B = 0, shift = 0, pad = 0;
        in >> rows >> A >> B;
        int dt = MUON_BF16, act = 0, dwt = -1;
        bool oi = false, bias = false, res = false, z = false, z8 = false, actout = false, add = false, acc = false,
             db = false, x8 = false, y8 = false, null = false, capture = false;
        while (in >> word) {
            if (word == "f32") dt = MUON_F32;
            else if (word == "oi") oi = true;
            else if (word == "bias") bias = true;
            else if (word == "res") res = true;
            else if (word == "z") z = true;
            else if (word == "z8") z8 = true;
            else if (word == "actout") actout = true;
            else if (word == "add") add = true;
            else if (word == "acc") acc = true;
            else if (word == "db") db = true;
            else if (word == "x8") x8 = true;
            else if (word == "y8") y8 = true;
            else if (word == "null") null = true;
            else if (word == "capture") capture = true;
            else if (word.rfind("act=", 0) == 0) act = std::stoi(word.substr(4));
            else if (word.rfind("dw=", 0) == 0) dwt = std::stoi(word.substr(3));
            else if (word.rfind("shift=", 0) == 0) shift = std::stoll(word.substr(6));
            else if (word.rfind("pad=", 0) == 0) pad = std::stoll(word.substr(4));
            else return 2;
        }
        const int es = dt == MUON_BF16 ? 2 : 4;
        uintptr_t next = uintptr_t(1) << 40;
        auto mat = [&](int size, bool per_row = true) {
            next += uintptr_t(1) << 36;
            return null && per_row ? nullptr : reinterpret_cast<void*>(next + uintptr_t(shift) * uintptr_t(size));
        };
        auto vec = [&](int size) { return mat(size, false); };
        auto rowvec = [&] { return static_cast<float*>(mat(4)); };
        auto q8 = [&](int64_t cols) {
            return muon_act8{static_cast<int8_t*>(mat(1)), static_cast<uint8_t*>(mat(1)), cols + pad, (cols + 31) / 32 + pad};
        };
        void* stream = reinterpret_cast<void*>(uintptr_t(capture ? 1 : 0));
        muon_status st = MUON_ERR_INVALID_ARG;
        emu_log.clear();
        if (op == "ln") {
            muon_layernorm_args a{};
            a.x = mat(es), a.y = mat(es), a.gain = vec(es), a.rows = rows, a.cols = A, a.ld_x = a.ld_y = A + pad;
            a.dtype = a.param_dtype = dt, a.eps = 1e-5f, a.mean = rowvec(), a.rstd = rowvec();
            if (bias) a.bias = vec(es);
            if (y8) a.y8 = q8(A);
            st = muon_layernorm_forward(h, &a, stream);
        } else if (op == "lngrad") {
            muon_layernorm_grad_args a{};
            a.dy = mat(es), a.x = mat(es), a.dx = mat(es), a.gain = vec(es), a.dgain = vec(es), a.dbias = vec(es);
            a.mean = rowvec(), a.rstd = rowvec(), a.rows = rows, a.cols = A, a.ld_dy = a.ld_x = a.ld_dx = A + pad;
            a.dtype = a.param_dtype = dt, a.accumulate = acc;
            if (add) a.add = mat(es), a.ld_add = A + pad;
            st = muon_layernorm_backward(h, &a, stream);
        } else if (op == "fwd") {
            muon_linear_args a{};
            a.x = mat(es), a.w = vec(es), a.y = mat(es), a.rows = rows, a.in = A, a.out = B;
            a.ld_x = A + pad, a.ld_w = (oi ? A : B) + pad, a.ld_y = B + pad, a.dtype = a.bias_dtype = dt;
            a.activation = act, a.w_layout = oi;
            if (bias) a.bias = vec(es);
            if (res) a.residual = mat(es), a.ld_residual = B + pad;
            if (z) a.z = mat(es), a.ld_z = B + pad;
            if (z8) a.z8 = q8(B);
            st = muon_linear_forward(h, &a, stream);
        } else if (op == "dx") {
            muon_linear_grad_input_args a{};
            a.dy = mat(es), a.w = vec(es), a.dx = mat(es), a.rows = rows, a.in = A, a.out = B;
            a.ld_dy = B + pad, a.ld_w = (oi ? A : B) + pad, a.ld_dx = A + pad, a.dtype = dt, a.activation = act;
            a.w_layout = oi;
            if (z) a.z = mat(es), a.ld_z = A + pad;
            if (z8) a.z8 = q8(A);
            if (actout) a.act_out = mat(es), a.ld_act_out = A + pad;
            if (add) a.add = mat(es), a.ld_add = A + pad;
            st = muon_linear_grad_input(h, &a, stream);
        } else if (op == "dw") {
            muon_linear_grad_weight_args a{};
            a.dy = mat(es), a.rows = rows, a.in = A, a.out = B, a.ld_dy = B + pad, a.ld_dw = (oi ? A : B) + pad;
            a.dtype = dt, a.dw_dtype = a.db_dtype = dwt < 0 ? dt : dwt, a.w_layout = oi, a.accumulate = acc;
            a.dw = vec(a.dw_dtype == MUON_BF16 ? 2 : 4);
            if (x8) a.x8 = q8(A);
            else a.x = mat(es), a.ld_x = A + pad;
            if (db) a.db = vec(4);
            st = muon_linear_grad_weight(h, &a, stream);
        } else if (op == "enc" || op == "dec") {
            void* x = mat(es);
            const muon_act8 q = q8(A);
            st = op == "enc" ? muon_act_encode(h, x, rows, A, A + pad, dt, &q, stream)
                             : muon_act_decode(h, &q, x, rows, A, A + pad, dt, stream);
        } else {
            return 2;
        }
        std::string err = muon_last_error(h);
        for (char& c : err)
            if (c == '"' || c == '\\') c = ' ';
        std::cout << "{\"status\": " << int(st) << ", \"error\": \"" << err << "\", \"workspace\": "
                  << muon_workspace_bytes(h) << ", \"launches\": [" << emu_log << "]}\n";
    }
    muon_destroy(h);
    return 0;
}
