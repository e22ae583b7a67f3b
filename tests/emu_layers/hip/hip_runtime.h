// Test infrastructure: the CPU stand-in of HIP (tests/emu) with what the layer
// operators' kernels use besides: two-dimensional grids, buffer loads into LDS
// with the hardware's range check, lane swaps (no-ops: one thread at a time)
// and the hardware's exp and reciprocal.
#pragma once
#include "../../emu/hip/hip_runtime.h"

#undef hipLaunchKernelGGL
template <class F, class... A>
inline void emu_launch2(const char* name, F f, dim3 g, dim3 b, A... a) {
    ++emu_launches;
    if (emu_verbose) std::fprintf(stderr, "launch %s grid %u x %u block %u\n", name, g.x, g.y, b.x);
    gridDim = g;
    blockDim = b;
    for (unsigned by = 0; by < g.y; ++by)
        for (unsigned bx = 0; bx < g.x; ++bx)
            for (unsigned tx = 0; tx < b.x; ++tx) {
                blockIdx = {bx, by, 0};
                threadIdx = {tx, 0, 0};
                f(a...);
            }
}
#define hipLaunchKernelGGL(K, G, B, SH, ST, ...) emu_launch2(#K, K, G, B, __VA_ARGS__)

inline uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
inline float emu_exp2(float x) { return std::exp2(x); }
#define __builtin_amdgcn_exp2f emu_exp2
#define __builtin_amdgcn_rcpf(x) (1.f / (x))
inline float emu_med3(float a, float b, float c) { return std::fmax(b, std::fmin(a, c)); }
#define __builtin_amdgcn_fmed3f emu_med3
typedef unsigned emu_u2 __attribute__((ext_vector_type(2)));
#define __builtin_amdgcn_permlane32_swap(a, b, x, y) (emu_u2{(a), (b)})
#define __builtin_amdgcn_permlane16_swap(a, b, x, y) (emu_u2{(a), (b)})
#define __builtin_amdgcn_s_barrier() ((void)0)
#define __builtin_amdgcn_s_setprio(x) ((void)0)
#define __builtin_amdgcn_sched_barrier(x) ((void)0)

// raw buffer: words 0-1 the base, word 2 the size in bytes; a lane past it stores zeros
inline char* emu_lds;   // the running kernel's LDS: its addresses count from there
inline uint32_t emu_lds_base(char* smem) {
    emu_lds = smem;
    return 0;
}
template <class V>
inline void emu_buffer_to_lds(V buf, uint32_t voff, uint32_t lds) {
    char* dst = emu_lds + lds + (threadIdx.x & 63) * 16;
    if (voff >= uint32_t(buf[2])) {
        std::memset(dst, 0, 16);
        return;
    }
    const uint64_t base = uint64_t(uint32_t(buf[0])) | (uint64_t(uint32_t(buf[1])) << 32);
    std::memcpy(dst, reinterpret_cast<const char*>(base) + voff, 16);
}
#define MUON_LDS_BASE emu_lds_base
#define MUON_BUFFER_TO_LDS emu_buffer_to_lds
