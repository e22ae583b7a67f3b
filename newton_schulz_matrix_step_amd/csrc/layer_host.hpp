// Host code that the layer operators' entry points share: argument checks,
// workspaces, the device guard.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <new>
#include <vector>

#pragma GCC visibility push(default)
#include "../../include/muon.h"
#pragma GCC visibility pop
#include "layer_internal.hpp"

namespace muon {

constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = (int64_t(1) << 31) - 1;

inline muon_status fail(HandleBase* h, muon_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    h->err = buf;
    return st;
}

inline muon_status hip_fail(HandleBase* h, hipError_t e, const char* what) {
    return fail(h, MUON_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// The handle's device for a scope; the calls are short, so a device that is
// current already is left alone.
struct DeviceGuard {
    int old = -1;
    bool ok = true, set = false;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&old) != hipSuccess) old = -1;
        if (old != dev) {
            set = true;
            ok = hipSetDevice(dev) == hipSuccess;
        }
    }
    ~DeviceGuard() {
        if (set && old >= 0) (void)hipSetDevice(old);
    }
};

// The handle's workspaces for these operators.  A block that has been handed
// out may be read by a captured graph, so no block is freed before the handle:
// a call takes the smallest one that is large enough, and only when there is
// none is a new one allocated, of twice the largest or more.  So the blocks of
// calls that grow a little at a time are few, and all of them together hold
// less than four times what the largest call needs (the last block less than
// twice that, the ones before it less than the last).  Where twice the largest
// cannot be had, the new block is what the call needs.
struct LayerState : HandleExt {
    struct Block {
        void* p;
        size_t bytes;
    };
    std::vector<Block> blocks;
    ~LayerState() override {
        for (Block& b : blocks) (void)hipFree(b.p);
    }
    int64_t workspace_bytes() const override {
        int64_t n = 0;
        for (const Block& b : blocks) n += int64_t(b.bytes);
        return n;
    }
};

inline muon_status workspace(HandleBase* h, size_t bytes, hipStream_t stream, void** out) {
    *out = nullptr;
    if (bytes == 0) return MUON_OK;
    if (!h->layers) {
        h->layers.reset(new (std::nothrow) LayerState());
        if (!h->layers) return fail(h, MUON_ERR_OOM, "workspace allocation failed");
    }
    LayerState& st = static_cast<LayerState&>(*h->layers);
    const LayerState::Block* best = nullptr;
    size_t largest = 0;
    for (const LayerState::Block& b : st.blocks) {
        largest = std::max(largest, b.bytes);
        if (b.bytes >= bytes && (!best || b.bytes < best->bytes)) best = &b;
    }
    if (best) {
        *out = best->p;
        return MUON_OK;
    }
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    const hipError_t e = hipStreamIsCapturing(stream, &cs);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return hip_fail(h, e, "hipStreamIsCapturing");
    }
    if (cs != hipStreamCaptureStatusNone)
        return fail(h, MUON_ERR_INVALID_ARG,
                    "a call captured into a HIP graph must first run once outside capture with the same sizes "
                    "(its workspace is then resident)");
    if (h->flags & MUON_INIT_FAIL_ALLOC)
        return fail(h, MUON_ERR_OOM, "workspace allocation failed (forced by MUON_INIT_FAIL_ALLOC)");
    auto mib = [](size_t n) { return (n + 0xFFFFFu) & ~size_t(0xFFFFF); };
    LayerState::Block b{nullptr, mib(std::max(bytes, 2 * largest))};
    try {
        st.blocks.reserve(st.blocks.size() + 1);
    } catch (const std::bad_alloc&) {
        return fail(h, MUON_ERR_OOM, "workspace allocation failed");
    }
    bool got = hipMalloc(&b.p, b.bytes) == hipSuccess;
    if (!got && b.bytes > mib(bytes)) {
        (void)hipGetLastError();
        b.bytes = mib(bytes);
        got = hipMalloc(&b.p, b.bytes) == hipSuccess;
    }
    if (!got) {
        (void)hipGetLastError();
        return fail(h, MUON_ERR_OOM, "workspace allocation of %.3f GB failed", double(b.bytes) / 1e9);
    }
    st.blocks.push_back(b);
    *out = b.p;
    return MUON_OK;
}

inline bool known_dtype(int32_t d) { return d == MUON_BF16 || d == MUON_F32; }
inline int esize(int32_t d) { return d == MUON_BF16 ? 2 : 4; }
inline int32_t dt_code(int32_t d) { return d == MUON_BF16 ? 0 : 1; }
inline bool aligned(const void* p, uintptr_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

// 16-byte vectors are legal on every row of the matrix.
inline bool rows_vec(const void* p, int64_t ld, int32_t dtype) { return aligned(p, 16) && ld * esize(dtype) % 16 == 0; }

struct Check {   // collects the first complaint
    HandleBase* h;
    muon_status st = MUON_OK;
    void need(bool ok, const char* fmt, ...) {
        if (ok || st != MUON_OK) return;
        char buf[256];
        va_list ap;
        va_start(ap, fmt);
        vsnprintf(buf, sizeof buf, fmt, ap);
        va_end(ap);
        st = fail(h, MUON_ERR_INVALID_ARG, "%s", buf);
    }
    void dtype(int32_t d, const char* what) {
        if (known_dtype(d) || st != MUON_OK) return;
        st = fail(h, MUON_ERR_DTYPE, "%s: unknown dtype %d", what, d);
    }
    void size(int64_t v, int64_t lo, int64_t hi, const char* what) {
        need(v >= lo && v <= hi, "%s %lld outside %lld..%lld", what, (long long)v, (long long)lo, (long long)hi);
    }
    // a matrix of `cols` columns, or an absent optional one
    void matrix(const void* p, int64_t ld, int64_t cols, int32_t dtype, const char* what) {
        if (!p) return;
        need(ld >= cols && ld <= kMaxLd, "%s: leading dimension %lld outside %lld..%lld", what, (long long)ld,
             (long long)cols, (long long)kMaxLd);
        need(aligned(p, uintptr_t(known_dtype(dtype) ? esize(dtype) : 1)), "%s: address not aligned to its elements", what);
    }
    void vector(const void* p, int32_t dtype, const char* what) {
        if (p) need(aligned(p, uintptr_t(known_dtype(dtype) ? esize(dtype) : 1)), "%s: address not aligned to its elements", what);
    }
    void act8(const muon_act8& q, int64_t cols, const char* what) {
        if (!q.codes) {
            need(!q.exponents, "%s: exponents without codes", what);
            return;
        }
        need(q.exponents != nullptr, "%s: codes without exponents", what);
        need(q.ld_codes >= cols && q.ld_codes <= kMaxLd, "%s: ld_codes %lld outside %lld..%lld", what,
             (long long)q.ld_codes, (long long)cols, (long long)kMaxLd);
        const int64_t g = (cols + kAct8Group - 1) / kAct8Group;
        need(q.ld_exponents >= g && q.ld_exponents <= kMaxLd, "%s: ld_exponents %lld outside %lld..%lld", what,
             (long long)q.ld_exponents, (long long)g, (long long)kMaxLd);
        need(static_cast<const void*>(q.codes) != static_cast<const void*>(q.exponents), "%s: codes alias exponents", what);
    }
    // no output may be an input or another output
    void distinct(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
        for (auto o = outs.begin(); o != outs.end(); ++o) {
            if (!*o) continue;
            for (auto p = o + 1; p != outs.end(); ++p) need(*o != *p, "two outputs alias");
            for (const void* in : ins) need(*o != in, "an output aliases an input");
        }
    }
};

inline Act8View act8_view(const muon_act8& q) {
    Act8View v{q.codes, q.exponents, q.ld_codes, q.ld_exponents, 0};
    v.vec = q.codes && aligned(q.codes, 8) && q.ld_codes % 8 == 0;
    return v;
}

// A call's common beginning: handle and struct present, device selected.
#define LAYER_ENTER(H, ARGS)                                                     \
    if (!(H)) return MUON_ERR_INVALID_ARG;                                       \
    HandleBase* h = handle_base(H);                                              \
    h->err.clear();                                                              \
    if (!(ARGS)) return fail(h, MUON_ERR_INVALID_ARG, #ARGS " is NULL");         \
    Check ck{h}

// Operand tiles are addressed by 32-bit byte offsets from the tile's first
// element: 256 rows, or 64 rows of k, must stay within 2^31 bytes.
inline bool tile_offsets_fit(int64_t ld, int64_t rows, int es) { return ld * es * rows + 1024 < (int64_t(1) << 31); }

// Whether 16-byte chunks of an operand are aligned and either whole or absent:
// along its contiguous dimension (k for a row-contiguous operand).
inline bool operand_dma(const void* p, int64_t ld, int64_t contiguous, bool kc, int es) {
    return aligned(p, 16) && ld * es % 16 == 0 && contiguous * es % 16 == 0 && tile_offsets_fit(ld, kc ? 256 : 64, es);
}

// No exception (an allocation of the host's that fails) leaves a C entry.
template <class F>
muon_status guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return MUON_ERR_OOM;
    }
}

}  // namespace muon
