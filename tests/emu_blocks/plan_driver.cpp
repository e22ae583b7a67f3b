// Test infrastructure: prints the tile edge, LDS depth and split that the library
// plans for gated products.  One per line of stdin: KIND (fwd dh dx dw) ROWS IN
// HIDDEN DTYPE (0 bf16, 1 float32) LAYOUT (0 in x out, 1 out x in).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <iostream>
#include <string>

#include "layer_internal.hpp"

emu_idx threadIdx, blockIdx;
dim3 gridDim, blockDim;
long emu_launches = 0;
int emu_verbose = 0;

int main() {
    std::string kind;
    long rows, in, hid, dt, oi;
    while (std::cin >> kind >> rows >> in >> hid >> dt >> oi) {
        muon::GatedArgs a;
        std::memset(&a, 0, sizeof a);
        a.dt = int(dt);
        a.a_dma = a.b_dma = a.a_kc = 1;
        a.M = rows;
        if (kind == "fwd") a.kind = muon::LIN_GATED, a.pair = muon::PAIR_COLS, a.N = hid, a.K = in, a.b_kc = oi;
        else if (kind == "dh") a.kind = muon::LIN_GATED_DH, a.N = hid, a.K = in, a.b_kc = !oi;
        else if (kind == "dx") a.kind = muon::LIN_DX, a.pair = muon::PAIR_K, a.N = in, a.K = hid, a.b_kc = !oi;
        else a.kind = muon::LIN_DW, a.pair = muon::PAIR_OUT, a.M = in, a.N = hid, a.K = rows, a.a_kc = 0, a.out_trans = oi;
        muon::plan_gated(a);
        std::printf("%d %d %d\n", a.tile, a.deep, a.splits);
    }
}
