// Test infrastructure: the epilogues' activations (layer_device.hpp) built for
// the host.  Reads lines "ACT Z" (1 GELU, 2 squared ReLU; Z as C's strtof takes
// it) and prints the forward value, then the value and derivative that the
// backward pass computes.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>

#include "layer_device.hpp"

emu_idx threadIdx, blockIdx;
dim3 gridDim, blockDim;
long emu_launches = 0;
int emu_verbose = 0;

int main() {
    int act;
    char z[64];
    while (std::scanf("%d %63s", &act, z) == 2) {
        const float x = std::strtof(z, nullptr);
        float v, d;
        muon::layer::act_both(x, act, v, d);
        std::printf("%.9g %.9g %.9g\n", muon::layer::act_value(x, act), v, d);
    }
    return 0;
}
