// Test infrastructure: the CPU stand-in of HIP (tests/emu_layers) with launches
// written down instead of run, so that calls of any size can be made with
// addresses that nothing reads; allocations over a limit fail, and a stream
// other than null counts as capturing.
#pragma once
#include "../../emu_layers/hip/hip_runtime.h"

#include <string>
#include <type_traits>
#include <utility>

#undef hipLaunchKernelGGL
inline std::string emu_log;          // the launches of the current call, as JSON objects
inline size_t emu_limit = ~size_t(0);

template <class A, class = void>
struct emu_is_product : std::false_type {};
template <class A>
struct emu_is_product<A, std::void_t<decltype(std::declval<A>().splits), decltype(std::declval<A>().out_trans)>>
    : std::true_type {};

// The sizes of a product's arguments (muon::LinArgs); nothing of other kernels'.
template <class A>
inline void emu_describe(const A& a) {
    if constexpr (emu_is_product<A>::value) {
        char b[256];
        std::snprintf(b, sizeof b,
                      ", \"kind\": %d, \"dt\": %d, \"tile\": %d, \"splits\": %d, \"deep\": %d, \"a_dma\": %d, \"b_dma\": %d, "
                      "\"codes\": %d, \"a_ld\": %lld, \"b_ld\": %lld, \"act_stream\": %d",
                      a.kind, a.dt, a.tile, a.splits, a.deep, a.a_dma, a.b_dma, a.a_exps ? 1 : 0, (long long)a.a_ld,
                      (long long)a.b_ld, a.act_stream);
        emu_log += b;
    }
}
template <class A0, class... A>
inline void emu_record(const char* name, dim3 g, dim3 b, const A0& a0, const A&...) {
    ++emu_launches;
    std::string s = name;
    for (char& c : s)
        if (c == '"' || c == '\\') c = ' ';
    emu_log += emu_log.empty() ? "{" : ", {";
    emu_log += "\"kernel\": \"" + s + "\", \"grid\": " + std::to_string(g.x) + ", \"grid_y\": " + std::to_string(g.y) +
               ", \"block\": " + std::to_string(b.x);
    emu_describe(a0);
    emu_log += "}";
}
#define hipLaunchKernelGGL(K, G, B, SH, ST, ...) emu_record(#K, G, B, __VA_ARGS__)

template <class T>
inline hipError_t emu_limited_malloc(T** p, size_t n) {
    if (n > emu_limit) {
        *p = nullptr;
        return 2;
    }
    return hipMalloc(p, n < 64 ? n : 64);   // only its address is used
}
#define hipMalloc emu_limited_malloc
inline hipError_t emu_capturing(hipStream_t s, hipStreamCaptureStatus* st) {
    *st = s ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}
#define hipStreamIsCapturing emu_capturing
